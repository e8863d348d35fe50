"""Host-side checks of the operators around the convolution (no GPU needed):
every refusal comes before any device work, so the calls below, on addresses
that nothing may touch, return it on any machine."""
import ctypes

import pytest

from causal_conv3d_video_b200 import ccv3d
from causal_conv3d_video_b200.ccv3d import (CCV3D_ERR_ALIAS, CCV3D_ERR_ALIGNMENT,
                                            CCV3D_ERR_INVALID, CCV3D_ERR_SCRATCH_LIMIT,
                                            CCV3D_ERR_UNSUPPORTED, CCV3D_OK)

A = 1 << 24  # buffers 16 MB apart


def _addr(i):
    return (i + 1) * A


NORM = ("h", "b", "gate", "post_w", "post_bias", "pre_w", "pre_bias", "h_out", "y")


def norm_forward(desc=None, **over):
    d = dict(rows=64, C=96, pre="rms", post="rms", act="silu", gate_rows=64)
    a = {k: _addr(i) for i, k in enumerate(NORM)}
    for k, v in over.items():
        (a if k in a else d)[k] = v
    desc = ccv3d.make_norm_desc(**d) if desc is None else desc
    return ccv3d.ccv3d_norm_forward(desc, *[a[k] for k in NORM], stream=0, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), CCV3D_ERR_INVALID), (dict(C=0), CCV3D_ERR_INVALID),
    (dict(C=8193), CCV3D_ERR_UNSUPPORTED), (dict(rows=1 << 60), CCV3D_ERR_UNSUPPORTED),
    (dict(eps=0.0), CCV3D_ERR_INVALID), (dict(eps=float("nan")), CCV3D_ERR_INVALID),
    (dict(eps=float("inf")), CCV3D_ERR_INVALID), (dict(scale=float("nan")), CCV3D_ERR_INVALID),
    (dict(gate_rows=0), CCV3D_ERR_INVALID), (dict(gate_rows=63), CCV3D_ERR_INVALID),
    (dict(h=None), CCV3D_ERR_INVALID), (dict(h_out=None), CCV3D_ERR_INVALID),
    (dict(y=None), CCV3D_ERR_INVALID), (dict(b=None), CCV3D_ERR_INVALID),
    (dict(post="none"), CCV3D_ERR_INVALID),               # weights of a norm that is not there
    (dict(pre="none"), CCV3D_ERR_INVALID),                # y without its norm
    (dict(h=_addr(0) + 2), CCV3D_ERR_ALIGNMENT), (dict(pre_w=_addr(5) + 8), CCV3D_ERR_ALIGNMENT),
    (dict(y=_addr(0)), CCV3D_ERR_ALIAS), (dict(y=_addr(1) + 16), CCV3D_ERR_ALIAS),
    (dict(h_out=_addr(0) + 192), CCV3D_ERR_ALIAS),        # h shifted by one row
    (dict(h_out=_addr(1)), CCV3D_ERR_ALIAS), (dict(y=_addr(7)), CCV3D_ERR_ALIAS),
    (dict(y=_addr(5)), CCV3D_ERR_ALIAS),
    (dict(rows=0), CCV3D_OK),
])
def test_norm_forward_refusals(over, status):
    assert norm_forward(**over) == status


def test_norm_unknown_kinds():
    for field, status in (("dtype", CCV3D_ERR_UNSUPPORTED), ("pre", CCV3D_ERR_UNSUPPORTED),
                          ("post", CCV3D_ERR_UNSUPPORTED), ("act", CCV3D_ERR_UNSUPPORTED)):
        for value in (7, -1):
            desc = ccv3d.make_norm_desc(rows=64, C=96)
            setattr(desc, field, value)
            assert norm_forward(desc) == status
            assert ccv3d.ccv3d_norm_workspace(desc) == 0
    assert ccv3d.lib.ccv3d_norm_forward(None, *[None] * 10) == CCV3D_ERR_INVALID
    assert ccv3d.lib.ccv3d_norm_workspace(None) == 0


BACK = ("h_out", "b", "gate", "post_w", "post_bias", "pre_w", "pre_bias", "dy", "dh_out", "dh",
        "db", "dgate", "dpost_w", "dpost_bias", "dpre_w", "dpre_bias", "ws")


@pytest.mark.parametrize("over,status", [
    (dict(h_out=None), CCV3D_ERR_INVALID), (dict(dy=None), CCV3D_ERR_INVALID),
    (dict(gate=None), CCV3D_ERR_INVALID),                 # dgate of no gate
    (dict(post_bias=None), CCV3D_ERR_INVALID), (dict(pre_w=None), CCV3D_ERR_INVALID),
    (dict(b=None), CCV3D_ERR_INVALID), (dict(gate_rows=7), CCV3D_ERR_INVALID),
    (dict(ws=None), CCV3D_ERR_INVALID), (dict(ws_bytes=100), CCV3D_ERR_SCRATCH_LIMIT),
    (dict(dh=_addr(8)), CCV3D_ERR_ALIAS), (dict(db=_addr(1)), CCV3D_ERR_ALIAS),
    (dict(ws=_addr(9)), CCV3D_ERR_ALIAS), (dict(dpre_w=_addr(13)), CCV3D_ERR_ALIAS),
    (dict(dh=_addr(9) + 4), CCV3D_ERR_ALIGNMENT), (dict(ws=_addr(16) + 4), CCV3D_ERR_ALIGNMENT),
])
def test_norm_backward_refusals(over, status):
    d = dict(rows=64, C=96, pre="rms", post="rms", act="silu", gate_rows=32)
    a = {k: _addr(i) for i, k in enumerate(BACK)}
    n = over.pop("ws_bytes", None) if "ws_bytes" in over else None
    for k, v in over.items():
        (a if k in a else d)[k] = v
    desc = ccv3d.make_norm_desc(**d)
    need = ccv3d.ccv3d_norm_workspace(desc)
    rc = ccv3d.lib.ccv3d_norm_backward(ctypes.byref(desc), *[a[k] for k in BACK],
                                       need if n is None else n, None)
    assert rc == status
    if n is not None:
        over["ws_bytes"] = n


POINT = ("x", "w", "bias", "residual", "out", "pre", "ws")


@pytest.mark.parametrize("over,status", [
    (dict(pixels=-1), CCV3D_ERR_INVALID), (dict(Cin=0), CCV3D_ERR_INVALID),
    (dict(Cout=0), CCV3D_ERR_INVALID), (dict(Cin=65537), CCV3D_ERR_UNSUPPORTED),
    (dict(Cout=65537), CCV3D_ERR_UNSUPPORTED), (dict(pixels=1 << 31), CCV3D_ERR_UNSUPPORTED),
    (dict(x=None), CCV3D_ERR_INVALID), (dict(w=None), CCV3D_ERR_INVALID),
    (dict(out=None), CCV3D_ERR_INVALID), (dict(x=_addr(0) + 2), CCV3D_ERR_ALIGNMENT),
    (dict(bias=_addr(2) + 2), CCV3D_ERR_ALIGNMENT), (dict(out=_addr(0)), CCV3D_ERR_ALIAS),
    (dict(out=_addr(3) + 192), CCV3D_ERR_ALIAS),          # the residual shifted by a row
    (dict(pre=_addr(4)), CCV3D_ERR_ALIAS), (dict(pre=_addr(3)), CCV3D_ERR_ALIAS),
    (dict(pixels=0), CCV3D_OK),
])
def test_pointwise_forward_refusals(over, status):
    d = dict(pixels=64, Cin=192, Cout=96, act="silu")
    a = {k: _addr(i) for i, k in enumerate(POINT)}
    for k, v in over.items():
        (a if k in a else d)[k] = v
    desc = ccv3d.make_pointwise_desc(**d)
    rc = ccv3d.lib.ccv3d_pointwise_forward(ctypes.byref(desc), *[a[k] for k in POINT], A // 2, None)
    assert rc == status


PBACK = ("x", "w", "pre", "dout", "dx", "dw", "dbias", "ws")


@pytest.mark.parametrize("over,status", [
    (dict(dout=None), CCV3D_ERR_INVALID), (dict(x=None), CCV3D_ERR_INVALID),
    (dict(w=None), CCV3D_ERR_INVALID), (dict(pre=None), CCV3D_ERR_INVALID),
    (dict(act="none"), CCV3D_ERR_INVALID),                # pre of no activation
    (dict(ws=None), CCV3D_ERR_INVALID), (dict(ws_bytes=16), CCV3D_ERR_SCRATCH_LIMIT),
    (dict(dx=_addr(0)), CCV3D_ERR_ALIAS), (dict(dw=_addr(1)), CCV3D_ERR_ALIAS),
    (dict(dbias=_addr(7)), CCV3D_ERR_ALIAS), (dict(dx=_addr(4) + 8), CCV3D_ERR_ALIGNMENT),
])
def test_pointwise_backward_refusals(over, status):
    over = dict(over)
    n = over.pop("ws_bytes", A // 2)
    d = dict(pixels=64, Cin=192, Cout=96, act="silu")
    a = {k: _addr(i) for i, k in enumerate(PBACK)}
    for k, v in over.items():
        (a if k in a else d)[k] = v
    desc = ccv3d.make_pointwise_desc(**d)
    rc = ccv3d.lib.ccv3d_pointwise_backward(ctypes.byref(desc), *[a[k] for k in PBACK], n, None)
    assert rc == status


def test_pointwise_unknown_kinds():
    for field in ("dtype", "act"):
        desc = ccv3d.make_pointwise_desc(pixels=4, Cin=8, Cout=8)
        setattr(desc, field, 9)
        with pytest.raises(ccv3d.CCV3DError) as e:
            ccv3d.ccv3d_pointwise_workspace(desc)
        assert e.value.status == CCV3D_ERR_UNSUPPORTED
    assert ccv3d.lib.ccv3d_pointwise_workspace(None, None, None) == CCV3D_ERR_INVALID


def qdesc(**over):
    d = dict(N=1, H=4, W=6, C=96, ring_slots=3, format="int8")
    d.update(over)
    return ccv3d.make_qcache_desc(**d)


@pytest.mark.parametrize("over,status", [
    (dict(C=0), CCV3D_ERR_INVALID), (dict(H=0), CCV3D_ERR_INVALID), (dict(N=-1), CCV3D_ERR_INVALID),
    (dict(ring_slots=0), CCV3D_ERR_INVALID), (dict(C=65537), CCV3D_ERR_UNSUPPORTED),
    (dict(H=1 << 16, W=1 << 16), CCV3D_ERR_UNSUPPORTED),
])
def test_qcache_desc_refusals(over, status):
    with pytest.raises(ccv3d.CCV3DError) as e:
        ccv3d.ccv3d_qcache_sizes(qdesc(**over))
    assert e.value.status == status


def test_qcache_unknown_kinds():
    for field in ("dtype", "format"):
        desc = qdesc()
        setattr(desc, field, 3)
        with pytest.raises(ccv3d.CCV3DError) as e:
            ccv3d.ccv3d_qcache_sizes(desc)
        assert e.value.status == CCV3D_ERR_UNSUPPORTED


def test_qcache_sizes():
    assert ccv3d.ccv3d_qcache_sizes(qdesc()) == (3 * 24 * 96, 3 * 24 * 3)
    assert ccv3d.ccv3d_qcache_sizes(qdesc(format="e2m1", C=33)) == (3 * 24 * 17, 3 * 24 * 2)
    assert ccv3d.ccv3d_qcache_sizes(qdesc(N=0)) == (0, 0)


@pytest.mark.parametrize("args,status", [
    (dict(frames=4, T=4), CCV3D_ERR_INVALID),             # more than the ring holds
    (dict(frames=-1), CCV3D_ERR_INVALID), (dict(slot=3), CCV3D_ERR_INVALID),
    (dict(slot=-1), CCV3D_ERR_INVALID), (dict(first=1), CCV3D_ERR_INVALID),
    (dict(first=-1), CCV3D_ERR_INVALID), (dict(x=None), CCV3D_ERR_INVALID),
    (dict(codes=None), CCV3D_ERR_INVALID), (dict(scales=None), CCV3D_ERR_INVALID),
    (dict(x=_addr(0) + 2), CCV3D_ERR_ALIGNMENT), (dict(codes=_addr(0)), CCV3D_ERR_ALIAS),
    (dict(scales=_addr(1)), CCV3D_ERR_ALIAS), (dict(frames=0), CCV3D_OK),
])
def test_qcache_write_refusals(args, status):
    a = dict(x=_addr(0), T=2, first=0, frames=2, slot=0, codes=_addr(1), scales=_addr(2))
    a.update(args)
    assert ccv3d.ccv3d_qcache_write(qdesc(), a["x"], a["T"], a["first"], a["frames"], a["slot"],
                                    a["codes"], a["scales"], stream=0, check=False) == status


@pytest.mark.parametrize("args,status", [
    (dict(frames=4), CCV3D_ERR_INVALID), (dict(frames=-1), CCV3D_ERR_INVALID),
    (dict(head=3), CCV3D_ERR_INVALID), (dict(head=-1), CCV3D_ERR_INVALID),
    (dict(out=None), CCV3D_ERR_INVALID), (dict(codes=None), CCV3D_ERR_INVALID),
    (dict(out=_addr(1)), CCV3D_ERR_ALIAS), (dict(out=_addr(2) - 16), CCV3D_ERR_ALIAS),
    (dict(out=_addr(0) + 8), CCV3D_ERR_ALIGNMENT), (dict(frames=0), CCV3D_OK),
])
def test_qcache_read_refusals(args, status):
    a = dict(out=_addr(0), frames=2, head=0, codes=_addr(1), scales=_addr(2))
    a.update(args)
    assert ccv3d.ccv3d_qcache_read(qdesc(), a["codes"], a["scales"], a["head"], a["frames"],
                                   a["out"], stream=0, check=False) == status


@pytest.mark.parametrize("args,status", [
    (dict(C=64), CCV3D_ERR_INVALID), (dict(H=5), CCV3D_ERR_INVALID), (dict(N=2), CCV3D_ERR_INVALID),
    (dict(dtype="fp32"), CCV3D_ERR_INVALID), (dict(ring_slots=2), CCV3D_ERR_INVALID),
    (dict(head=3), CCV3D_ERR_INVALID), (dict(head=-1), CCV3D_ERR_INVALID),
    (dict(codes=None), CCV3D_ERR_INVALID), (dict(scales=None), CCV3D_ERR_INVALID),
    (dict(buf=None), CCV3D_ERR_INVALID), (dict(x=None), CCV3D_ERR_INVALID),
    (dict(codes=_addr(1) + 8), CCV3D_ERR_ALIGNMENT), (dict(buf=_addr(3) + 8), CCV3D_ERR_ALIGNMENT),
    (dict(codes=_addr(0)), CCV3D_ERR_ALIAS), (dict(scales=_addr(6)), CCV3D_ERR_ALIAS),
    (dict(buf=_addr(0)), CCV3D_ERR_ALIAS), (dict(buf=_addr(1)), CCV3D_ERR_ALIAS),
    (dict(buf=_addr(6)), CCV3D_ERR_ALIAS), (dict(pad=(0, 1)), CCV3D_ERR_INVALID),
])
def test_forward_qring_refusals(args, status):
    plan = ccv3d.Plan(ccv3d.make_desc(N=1, Cin=96, Cout=32, H=4, W=6, T_x=1, cache_len=2))
    a = dict(x=_addr(0), codes=_addr(1), scales=_addr(2), buf=_addr(3), w=_addr(4), bias=_addr(5),
             out=_addr(6), head=0, pad=(1, 1))
    d = {}
    for k, v in args.items():
        (a if k in a else d)[k] = v
    before = plan.stats()
    rc, nh = ccv3d.ccv3d_forward_qring(plan.handle, a["x"], qdesc(**d), a["codes"], a["scales"],
                                       a["head"], a["buf"], a["w"], a["bias"], a["out"], (1, 1),
                                       a["pad"], (1, 1, 1), stream=0, check=False)
    assert rc == status and nh == -1
    after = plan.stats()
    assert after["errors"] + after["unsupported"] == before["errors"] + before["unsupported"] + 1
    assert after["calls"] == 0


def test_binding_refuses_wrong_tensors():
    import torch
    desc = ccv3d.make_norm_desc(rows=4, C=8)
    good = torch.zeros(4, 8, dtype=torch.bfloat16)
    for h in (good.float(), torch.zeros(4, 9, dtype=torch.bfloat16),
              torch.zeros(8, 4, dtype=torch.bfloat16).t(), good):   # the last: not on a GPU
        with pytest.raises(ValueError):
            ccv3d.ccv3d_norm_forward(desc, h, None, None, None, None, None, None, None, A, stream=0)


def test_plan_forward_qring_checks_sizes():
    import torch
    plan = ccv3d.Plan(ccv3d.make_desc(N=1, Cin=96, Cout=32, H=4, W=6, T_x=1, cache_len=2))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    good = dict(x=bf(1, 1, 4, 6, 96), cache_buf=bf(1, 2, 4, 6, 96), w=bf(32, 3, 3, 3, 96),
                bias=bf(32), out=bf(1, 1, 4, 6, 32))
    for name in good:
        a = dict(good, **{name: bf(*good[name].shape)[..., :-8].contiguous()})
        with pytest.raises(ValueError, match=name):
            plan.forward_qring(a["x"], qdesc(), _addr(1), _addr(2), 0, a["cache_buf"], a["w"],
                               a["bias"], a["out"], stream=0)


def test_strerror_names_every_status():
    assert all(ccv3d.ccv3d_strerror(s) != "unknown status" for s in range(10))


def test_raw_workspace_addresses():
    """A workspace given as an address needs its size, and is then the call's."""
    nd = ccv3d.make_norm_desc(rows=64, C=96, post="rms", gate_rows=32)
    pd = ccv3d.make_pointwise_desc(pixels=64, Cin=192, Cout=96, act="silu")
    a = [_addr(i) for i in range(17)]
    for call, desc, n, need in (
            (ccv3d.ccv3d_norm_backward, nd, 17, ccv3d.ccv3d_norm_workspace(nd)),
            (ccv3d.ccv3d_pointwise_forward, pd, 7, 0),
            (ccv3d.ccv3d_pointwise_backward, pd, 8, ccv3d.ccv3d_pointwise_workspace(pd)[1])):
        with pytest.raises(ValueError, match="ws_bytes"):
            call(desc, *a[:n], stream=0, check=False)
        if need:
            assert call(desc, *a[:n], stream=0, check=False,
                        ws_bytes=need - 1) == CCV3D_ERR_SCRATCH_LIMIT
        b = list(a[:n])
        b[-2] = b[0]    # an output on an input: refused after the workspace's size
        assert call(desc, *b, stream=0, check=False, ws_bytes=need) == CCV3D_ERR_ALIAS


def test_forward_qring_checks_sizes():
    """The call itself, not Plan's method alone."""
    import torch
    plan = ccv3d.ccv3d_plan(ccv3d.make_desc(N=1, Cin=96, Cout=32, H=4, W=6, T_x=1, cache_len=2))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    good = dict(x=bf(1, 1, 4, 6, 96), cache_buf=bf(1, 2, 4, 6, 96), w=bf(32, 3, 3, 3, 96),
                bias=bf(32), out=bf(1, 1, 4, 6, 32))
    try:
        for name in good:
            for wrong in (good[name][..., :-8].contiguous(), torch.cat([good[name]] * 2)):
                if name == "cache_buf" and wrong.numel() > good[name].numel():
                    continue    # a scratch may be larger
                a = dict(good, **{name: wrong})
                with pytest.raises(ValueError, match=f"{name} has {wrong.numel()} elements"):
                    ccv3d.ccv3d_forward_qring(plan, a["x"], qdesc(), _addr(1), _addr(2), 0,
                                              a["cache_buf"], a["w"], a["bias"], a["out"], (1, 1),
                                              (1, 1), (1, 1, 1), stream=0)
    finally:
        ccv3d.ccv3d_destroy(plan)


@pytest.mark.parametrize("over", [
    dict(H=1 << 15, W=1 << 16), dict(N=1 << 16, ring_slots=1 << 15),
    dict(N=1 << 14, ring_slots=1 << 14, H=64, W=64, C=64)])
def test_qcache_stated_limits(over):
    with pytest.raises(ccv3d.CCV3DError) as e:
        ccv3d.ccv3d_qcache_sizes(qdesc(**over))
    assert e.value.status == CCV3D_ERR_UNSUPPORTED


def test_qcache_frames_of_a_call():
    """N * frames past what one call moves, for the write, the read and both in
    ccv3d_forward_qring; the last that it moves gets past that check."""
    N = 1 << 14
    d = qdesc(N=N, H=1, W=1, C=8, ring_slots=5)
    far = [(i + 1) << 32 for i in range(7)]
    for frames, status in ((4, CCV3D_ERR_UNSUPPORTED), (3, CCV3D_ERR_ALIAS)):
        assert ccv3d.ccv3d_qcache_write(d, far[0], 5, 0, frames, 0, far[1], far[1], stream=0,
                                        check=False) == status
        assert ccv3d.ccv3d_qcache_read(d, far[1], far[2], 0, frames, far[1], stream=0,
                                       check=False) == status
    for T_x, cache_len in ((4, 0), (1, 4)):
        plan = ccv3d.Plan(ccv3d.make_desc(N=N, Cin=8, Cout=8, H=1, W=1, T_x=T_x,
                                          cache_len=cache_len, cache_keep=4))
        rc, _ = ccv3d.ccv3d_forward_qring(plan.handle, far[0], d, far[1], far[2], 0, far[3], far[4],
                                          far[5], far[6], (1, 1), (1, 1), (1, 1, 1), stream=0,
                                          check=False)
        assert rc == CCV3D_ERR_UNSUPPORTED
