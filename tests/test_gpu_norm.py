"""ccv3d_norm_forward / ccv3d_norm_backward against their definition in 64 bits."""
import itertools

import pytest
import torch

from block_util import DT, HALF, ROW, act, close, d, guarded, norm
from causal_conv3d_video_b200 import ccv3d

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _case(rows, C, dtype, *, pre="rms", post="none", residual=False, gates=0, actk="none",
          bias=False, seed=0, scale=0.7, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, mean=0.0, std=1.0):
        return (torch.randn(s, device="cuda", generator=g) * std + mean).to(DT[dtype])

    s = dict(rows=rows, C=C, dtype=dtype, pre=pre, post=post, act=actk, scale=scale)
    s["h"] = rnd(rows, C, mean=0.3, std=1.5)
    s["b"] = rnd(rows, C, mean=-0.2) if residual else None
    s["gate"] = rnd(gates, C, mean=0.5) if gates else None
    use = lambda k: weights and k != "none"
    s["pre_w"] = rnd(C, mean=1.0, std=0.3) if use(pre) else None
    s["pre_bias"] = rnd(C, std=0.2) if use(pre) and bias else None
    s["post_w"] = rnd(C, mean=1.0, std=0.3) if use(post) else None
    s["post_bias"] = rnd(C, std=0.2) if use(post) and bias else None
    s["desc"] = ccv3d.make_norm_desc(rows=rows, C=C, pre=pre, post=post, act=actk, eps=EPS,
                                     scale=scale, gate_rows=rows // gates if gates else 0,
                                     dtype=dtype)
    s["rnd"] = rnd
    return s


def _forward(s, stream=None, h_out=None):
    y, ok_y = guarded((s["rows"], s["C"]), DT[s["dtype"]]) if s["pre"] != "none" else (None, None)
    if s["b"] is not None and h_out is None:
        h_out, ok_h = guarded((s["rows"], s["C"]), DT[s["dtype"]])
    else:
        ok_h = None
    ccv3d.ccv3d_norm_forward(s["desc"], s["h"], s["b"], s["gate"], s["post_w"], s["post_bias"],
                             s["pre_w"], s["pre_bias"], h_out, y, stream)
    torch.cuda.synchronize()
    for ok in (ok_y, ok_h):
        if ok:
            ok()
    return h_out, y


def _gate_rows(s):
    if s["gate"] is None:
        return torch.ones(1, s["C"], device="cuda", dtype=torch.float64)
    return d(s["gate"]).repeat_interleave(s["rows"] // s["gate"].shape[0], 0)


def _check_forward(s, h0=None, got=None):
    h_out, y = _forward(s) if got is None else got
    h = d(s["h"] if h0 is None else h0)
    half, row = HALF[s["dtype"]], ROW[s["dtype"]]
    if s["b"] is not None:
        p, _, _, mag = norm(d(s["b"]), s["post"], d(s["post_w"]), d(s["post_bias"]), EPS)
        g = s["scale"] * _gate_rows(s)
        want = h + g * p
        close(h_out, want, half * want.abs() + row * (h.abs() + g.abs() * mag), "h_out")
        h = d(h_out)
    if y is not None:
        u, _, _, mag = norm(h, s["pre"], d(s["pre_w"]), d(s["pre_bias"]), EPS)
        want = act(u, s["act"])
        # |act'| <= 1.13; a cancellation inside GELU's cubic costs a few more steps
        close(y, want, half * want.abs() + 2 * row * mag, "y")


SHAPES = [(1, 8), (1, 768), (3, 1), (5, 7), (33, 16), (17, 24), (64, 32), (129, 75), (100, 96),
          (31, 100), (77, 192), (50, 257), (40, 384), (9, 513), (23, 768), (21, 1000), (6, 1025),
          (5, 2048), (3, 4096), (2, 8185), (2, 8192)]
# enough rows for the tiles of rows (forward), odd ones for their ragged ends
TILED = [(5003, 1), (1009, 8), (777, 24), (2001, 32), (1500, 50), (3001, 75), (2300, 96), (701, 99),
         (1234, 160), (999, 192), (640, 257), (1111, 384), (401, 500), (333, 720), (600, 767),
         (500, 768), (700, 769), (350, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", SHAPES + TILED)
def test_forward_shapes(rows, C, dtype):
    _check_forward(_case(rows, C, dtype, actk="silu"))
    _check_forward(_case(rows, C, dtype, residual=True, gates=1, post="rms", actk="silu", seed=1))
    _check_forward(_case(rows, C, dtype, residual=True, post="layer", pre="layer", bias=True,
                         actk="gelu", seed=2))


@pytest.mark.parametrize("pre,post,gates,bias,weights", [
    (pre, post, g, b, w) for pre, post, g, b, w in itertools.product(
        ["none", "rms", "layer"], ["none", "rms", "layer"], [0, 1, 4, 60], [False, True],
        [True, False])])
def test_forward_forms(pre, post, gates, bias, weights):
    _check_forward(_case(60, 96, "bf16", pre=pre, post=post, residual=True, gates=gates, bias=bias,
                         weights=weights, actk="none"))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gate_rows_in_tiles(dtype):
    """Gate rows that change inside a tile, and groups of one row, three, many."""
    for rows, C, gates in [(1200, 96, 1200), (1200, 96, 400), (1300, 75, 13), (900, 193, 3),
                           (700, 768, 100), (1400, 40, 7)]:
        s = _case(rows, C, dtype, residual=True, gates=gates, post="rms", actk="silu", seed=gates)
        _check_forward(s)
        _check_backward(s)
        _check_forward(_case(rows, C, dtype, residual=True, gates=gates, post="layer", bias=True))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_fused_is_the_two_halves(dtype):
    """One call gives the bits of the post half followed by the pre half."""
    for rows, C in [(500, 96), (123, 75), (40, 1536)]:
        s = _case(rows, C, dtype, residual=True, gates=1, post="rms", actk="silu")
        h_out, y = _forward(s)
        a = dict(s, pre="none", pre_w=None, desc=ccv3d.make_norm_desc(
            rows=rows, C=C, pre="none", post="rms", eps=EPS, scale=0.7, gate_rows=rows,
            dtype=dtype))
        h2, _ = _forward(a)
        b = dict(s, h=h2, b=None, gate=None, post_w=None, desc=ccv3d.make_norm_desc(
            rows=rows, C=C, pre="rms", act="silu", eps=EPS, dtype=dtype))
        _, y2 = _forward(b)
        assert torch.equal(h_out, h2) and torch.equal(y, y2)


def test_stream_updated_in_place():
    s = _case(1000, 96, "bf16", residual=True, gates=1, post="rms", actk="silu")
    h0 = s["h"].clone()
    want = _forward(s)
    got = _forward(s, h_out=s["h"])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert not torch.equal(h0, s["h"])


def test_non_finite_rows_stay_alone():
    s = _case(64, 96, "bf16", residual=True, post="rms", actk="silu")
    s["h"][3, 5] = float("nan")
    s["b"][10, 7] = float("inf")
    s["h"][20] = 0
    s["b"][20] = 0
    h_out, y = _forward(s)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[3] = bad[10] = True
    assert torch.equal(y.isnan().any(1), bad)
    assert (y[20] == 0).all() and (h_out[20] == 0).all()


def _backward(s, want=None, stream=None, dh_out=True):
    C, dt = s["C"], DT[s["dtype"]]
    dy = s["rnd"](s["rows"], C) if s["pre"] != "none" else None
    dho = s["rnd"](s["rows"], C) if dh_out else None
    out, oks = {}, []
    for k in ("h", "b", "gate", "post_w", "post_bias", "pre_w", "pre_bias"):
        out["d" + k] = None
        if s[k] is not None and (want is None or k in want):
            out["d" + k], ok = guarded(tuple(s[k].shape), dt)
            oks.append(ok)
    n = ccv3d.ccv3d_norm_workspace(s["desc"])
    ws, ok = guarded((n,), torch.uint8, fill=9)
    oks.append(ok)
    ccv3d.ccv3d_norm_backward(s["desc"], s["h"], s["b"], s["gate"], s["post_w"], s["post_bias"],
                              s["pre_w"], s["pre_bias"], dy, dho, out["dh"], out["db"],
                              out["dgate"], out["dpost_w"], out["dpost_bias"], out["dpre_w"],
                              out["dpre_bias"], ws, stream)
    torch.cuda.synchronize()
    for ok in oks:
        ok()
    return dy, dho, {k: v for k, v in out.items() if v is not None}


def _check_backward(s, want=None, dh_out=True):
    dy, dho, got = _backward(s, want, dh_out=dh_out)
    half, row, rows = HALF[s["dtype"]], ROW[s["dtype"]], s["rows"]
    zero = torch.zeros(rows, s["C"], device="cuda", dtype=torch.float64)
    h = d(s["h"]).requires_grad_()
    leaves = {"dh": h}
    for k in ("b", "gate", "post_w", "post_bias", "pre_w", "pre_bias"):
        if s[k] is not None:
            leaves["d" + k] = d(s[k]).requires_grad_()
    L = lambda k: leaves.get("d" + k)
    # G: gradient of the stream; then the rest through the gate and the post norm
    mag_h = d(dho).abs() if dho is not None else zero
    G = d(dho) if dho is not None else zero
    terms = {}
    if dy is not None:
        u, n, rstd, mag = norm(h, s["pre"], L("pre_w"), L("pre_bias"), EPS)
        u_ = u.detach().requires_grad_()
        da, = torch.autograd.grad(act(u_, s["act"]).sum(), u_)
        du = d(dy) * da
        # the activation's second derivative is at most 1.1 (GELU), so an error
        # of u of `row` times its magnitude moves du by dy times that
        e_du = row * (du.abs() + d(dy).abs() * (1.2 * mag.detach() if s["act"] != "none" else 0))
        grads = torch.autograd.grad(u, [t for t in (h, L("pre_w"), L("pre_bias")) if t is not None],
                                    du, retain_graph=False)
        it = iter(grads)
        G = G + next(it)
        w = d(s["pre_w"]).abs() if s["pre_w"] is not None else 1.0
        n, rstd = n.detach(), rstd.detach()
        nmag = n.abs() + h.detach().abs().amax(1, keepdim=True) * rstd  # of the rows' own error
        dn, e_dn = du.abs() * w, e_du * w
        m1 = (dn * nmag).mean(1, keepdim=True)
        e_m1 = (e_dn * nmag + row * dn * nmag).mean(1, keepdim=True)
        mag_h = mag_h + rstd * (dn + nmag * m1 + dn.mean(1, keepdim=True))
        e_G = rstd * (e_dn + e_dn.mean(1, keepdim=True) + nmag * e_m1) + row * mag_h
        if L("pre_w") is not None:
            terms["dpre_w"] = (next(it), (e_du * nmag + row * du.abs() * nmag).sum(0))
        if L("pre_bias") is not None:
            terms["dpre_bias"] = (next(it), (e_du + row * du.abs()).sum(0))
    else:
        e_G = row * mag_h
    G = G.detach()
    if "dh" in got:
        close(got["dh"], G, half * G.abs() + e_G, "dh")
    if s["b"] is not None:
        b = L("b")
        p, m, rstd, mag = norm(b, s["post"], L("post_w"), L("post_bias"), EPS)
        gate = L("gate")
        per = gate.repeat_interleave(rows // gate.shape[0], 0) if gate is not None else 1.0
        keys = [k for k in ("db", "dgate", "dpost_w", "dpost_bias") if k in leaves]
        grads = dict(zip(keys, torch.autograd.grad(s["scale"] * per * p, [leaves[k] for k in keys],
                                                   G)))
        m, rstd, mag = m.detach(), rstd.detach(), mag.detach()
        sg = s["scale"] * (per.detach().abs() if gate is not None else 1.0)
        mm = m.abs() + (b.detach().abs().amax(1, keepdim=True) * rstd if s["post"] != "none" else 0)
        E = e_G + row * G.abs()  # of G and of each product with it
        grp = lambda t: t.view(gate.shape[0], -1, s["C"]).sum(1)
        if "dgate" in keys:
            terms["dgate"] = (grads["dgate"], s["scale"] * grp(E * mag + row * G.abs() * mag))
        if "dpost_w" in keys:
            terms["dpost_w"] = (grads["dpost_w"], (sg * (E * mm + row * G.abs() * mm)).sum(0))
        if "dpost_bias" in keys:
            terms["dpost_bias"] = (grads["dpost_bias"], (sg * E).sum(0))
        w = d(s["post_w"]).abs() if s["post_w"] is not None else 1.0
        dm, e_dm = sg * G.abs() * w, sg * E * w
        if s["post"] == "none":
            tol = e_dm + row * dm
        else:
            m1 = (dm * mm).mean(1, keepdim=True)
            e1 = (e_dm * mm + row * dm * mm).mean(1, keepdim=True)
            tol = rstd * (e_dm + e_dm.mean(1, keepdim=True) + mm * e1) + row * rstd * (
                dm + mm * m1 + dm.mean(1, keepdim=True))
        if "db" in got:
            close(got["db"], grads["db"], half * grads["db"].abs() + tol, "db")
    for k, (want_k, tol) in terms.items():
        if k in got:
            # a column is at most 2^9 sequential additions a thread here: 2^-15
            # of the terms' magnitudes, within the doubled allowance of each
            close(got[k], want_k, half * want_k.abs() + 4 * tol, k)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", SHAPES + TILED)
def test_backward_shapes(rows, C, dtype):
    _check_backward(_case(rows, C, dtype, actk="silu"))
    _check_backward(_case(rows, C, dtype, residual=True, gates=1, post="rms", actk="silu", seed=1))
    _check_backward(_case(rows, C, dtype, residual=True, post="layer", pre="layer", bias=True,
                          actk="gelu", seed=2))


@pytest.mark.parametrize("pre,post,gates,bias", [
    c for c in itertools.product(["none", "rms", "layer"], ["none", "rms", "layer"],
                                 [0, 1, 4, 60], [False, True])])
def test_backward_forms(pre, post, gates, bias):
    _check_backward(_case(60, 96, "fp32", pre=pre, post=post, residual=True, gates=gates,
                          bias=bias, actk="silu" if pre != "none" else "none"))


def test_backward_parts_and_long():
    s = _case(20000, 48, "bf16", residual=True, gates=8, post="rms", actk="silu", bias=True)
    _check_backward(s)
    for want in (["h"], ["b"], ["gate"], ["pre_w", "post_bias"], ["h", "b"]):
        _check_backward(s, want)
    _check_backward(_case(333, 40, "fp32", actk="gelu"), dh_out=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [96, 75, 1024, 1001, 5000])
def test_backward_without_the_stream(C, dtype):
    """Without a pre norm the stream's value is not read, and may be NULL."""
    cases = [_case(90, C, dtype, pre="none", post="rms", residual=True, gates=3, seed=5)
             for _ in range(3)]
    want = _backward(cases[0])[2]
    got = _backward(dict(cases[1], h=None))[2]
    assert set(got) == set(want) - {"dh"}
    assert all(torch.equal(got[k], want[k]) for k in got)
    _check_backward(cases[2])


def test_backward_same_bits_every_run():
    for C in (96, 75, 1536):
        s = _case(5000, C, "bf16", residual=True, gates=5, post="rms", actk="silu", bias=True)
        state = torch.Generator(device="cuda")
        runs = []
        for _ in range(2):
            s2 = _case(5000, C, "bf16", residual=True, gates=5, post="rms", actk="silu", bias=True)
            runs.append(_backward(s2)[2])
        del state, s
        assert all(torch.equal(runs[0][k], runs[1][k]) for k in runs[0])


def test_backward_against_differences():
    """Central differences of the forward definition in 64 bits, along random
    directions, against the fp32 kernel's gradients."""
    rows, C = 12, 40
    s = _case(rows, C, "fp32", pre="layer", post="rms", residual=True, gates=3, actk="gelu",
              bias=True)
    h_out, _ = _forward(s)
    back = dict(s, h=h_out)
    dy, dho, got = _backward(back)

    def loss(vals):
        g = vals["gate"].repeat_interleave(rows // 3, 0)
        p = norm(vals["b"], "rms", vals["post_w"], vals["post_bias"], EPS)[0]
        h = vals["h"] + s["scale"] * g * p
        y = act(norm(h, "layer", vals["pre_w"], vals["pre_bias"], EPS)[0], "gelu")
        return (y * d(dy)).sum() + (h * d(dho)).sum()

    base = {k: d(s[k]) for k in ("h", "b", "gate", "post_w", "post_bias", "pre_w", "pre_bias")}
    gen = torch.Generator(device="cuda").manual_seed(4)
    for k in base:
        v = torch.randn(base[k].shape, device="cuda", generator=gen, dtype=torch.float64)
        e = 1e-5
        up, dn = (loss({**base, k: base[k] + sgn * e * v}) for sgn in (1, -1))
        want = (up - dn) / (2 * e)
        have = (d(got["d" + k]) * v).sum()
        # differences: e^2 times third derivatives and 2^-53 / e of the loss; the
        # gradients: 2^-16 of the products' magnitudes (h_out was rounded to fp32)
        tol = 2.0 ** -16 * (d(got["d" + k]) * v).abs().sum() + 1e-6 * (1 + want.abs())
        assert abs(want - have) <= tol, (k, want, have)


def test_zero_rows():
    s = _case(0, 32, "bf16", residual=True, post="rms", bias=True)
    _forward(s)
    got = _backward(s)[2]
    assert all((got[k] == 0).all() for k in ("dpost_w", "dpost_bias", "dpre_w", "dpre_bias"))


def test_other_stream_and_graph():
    s = _case(3000, 96, "bf16", residual=True, gates=1, post="rms", actk="silu")
    want = _forward(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = _forward(s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    dy, dho, grads = _backward(s)
    n = ccv3d.ccv3d_norm_workspace(s["desc"])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = {k: torch.zeros_like(v) for k, v in grads.items()}
    h_out, y = torch.zeros_like(s["h"]), torch.zeros_like(s["h"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccv3d.ccv3d_norm_forward(s["desc"], s["h"], s["b"], s["gate"], s["post_w"], None,
                                 s["pre_w"], None, h_out, y)
        ccv3d.ccv3d_norm_backward(s["desc"], s["h"], s["b"], s["gate"], s["post_w"], None,
                                  s["pre_w"], None, dy, dho, outs["dh"], outs["db"],
                                  outs["dgate"], outs["dpost_w"], None, outs["dpre_w"], None, ws)
    for _ in range(2):
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[1]) and torch.equal(h_out, want[0])
        assert all(torch.equal(outs[k], grads[k]) for k in grads)


def test_far_rows():
    """Offsets past 2^31 bytes and elements: the last rows of a long call."""
    rows, C = 23_000_000, 96
    h = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    h[-5:] = torch.randn(5, C, device="cuda").bfloat16()
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(h)
    ccv3d.ccv3d_norm_forward(ccv3d.make_norm_desc(rows=rows, C=C, eps=EPS), h, None, None, None,
                             None, w, None, None, y)
    want, _, _, mag = norm(d(h[-5:]), "rms", d(w), None, EPS)
    close(y[-5:], want, HALF["bf16"] * want.abs() + ROW["bf16"] * mag, "y")
    assert int((y[:-5] != 0).sum()) == 0
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


@pytest.fixture(autouse=True)
def status_is_clean():
    """No call of a test left an error (a wait that ran out; in the checked build
    an address outside its buffer) in the library's status word."""
    yield
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", SHAPES + TILED)
def test_backward_layer_norms_without_biases(rows, C, dtype):
    """The form of layer norms alone: two column sums, and the rows' means."""
    _check_backward(_case(rows, C, dtype, residual=True, gates=1, pre="layer", post="layer",
                          actk="gelu", seed=3))
    _check_backward(_case(rows, C, dtype, residual=True, pre="layer", post="rms", actk="silu",
                          seed=4))
    _check_backward(_case(rows, C, dtype, pre="layer", weights=False, seed=5), dh_out=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,C", [(36, 776), (60, 1000), (24, 1025), (48, 2048), (12, 4104),
                                    (24, 5001), (12, 8185), (12, 8192), (3600, 1024)])
def test_wide_rows_with_several_gates(rows, C, dtype):
    for gates, pre, post, bias in [(3, "rms", "rms", False), (12, "layer", "layer", False),
                                   (2, "layer", "rms", True), (rows, "none", "layer", True)]:
        s = _case(rows, C, dtype, residual=True, gates=gates, pre=pre, post=post, bias=bias,
                  actk="silu" if pre != "none" else "none", seed=gates)
        _check_forward(s)
        _check_backward(s)
