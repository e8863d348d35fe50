"""The operators together, as a decoder's residual block uses them:
    norm + SiLU -> conv3d (quantised ring cache) -> norm + SiLU -> conv3d -> + 1x1x1 shortcut,
streamed frame by frame, against the same block in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from block_util import d, norm
from causal_conv3d_video_b200 import ccv3d
from causal_conv3d_video_b200.workloads import Conv
from parity_util import assert_close, oracle_params, plan_env
from test_gpu_qcache import quantise
from test_gpu_ring import RING_SIGS

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("Cin,Cout,H,W,T_x,dtype", [
    (32, 48, 9, 14, 1, "bf16"), (64, 64, 12, 20, 2, "bf16"), (24, 16, 5, 7, 1, "fp32")])
def test_forward_qring_streams(Cin, Cout, H, W, T_x, dtype, fmt):
    """Each call's output is ccv3d_forward's on the cache as read back (the
    oracle's on those values), and the ring holds the arriving frames' codes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, std=1.0: (torch.randn(s, device="cuda", generator=g) * std).to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    w, b = rnd(Cout, 3, 3, 3, Cin, std=(27 * Cin) ** -0.5), rnd(Cout, std=0.1)
    slots, keep = 2 + T_x, 2
    desc = ccv3d.make_qcache_desc(N=1, H=H, W=W, C=Cin, ring_slots=slots, format=fmt, dtype=dtype)
    codes, scales = ccv3d.alloc_qcache(desc)
    head, kept = 1, []        # kept: the frames the cache should hold, as read back
    for step in range(5):
        conv = Conv("s", Cin, Cout, H, W, T_x=T_x, cache_len=len(kept), dtype=dtype)
        plan = ccv3d.Plan(ccv3d.desc_for(conv))
        x = rnd(1, T_x, H, W, Cin)
        out, _ = plan.alloc_outputs("cuda")
        buf = rnd(1, len(kept), H, W, Cin) if kept else None
        head = plan.forward_qring(x, desc, codes, scales, head, buf, w, b, out)
        torch.cuda.synchronize()
        assert plan.status() == ccv3d.CCV3D_OK and plan.stats()["calls"] == 1
        cache = np.stack(kept, 1) if kept else None
        if kept:
            assert np.array_equal(_np(buf), cache)
        ref, _ = oracle.forward(oracle_params(conv), _np(x), cache, _np(w), _np(b))
        assert_close(_np(out), ref, dtype)
        kept = (kept + [quantise(_np(x)[:, t], fmt)[1] for t in range(T_x)])[-keep:]
        # the new head finds them again
        back = torch.empty(1, len(kept), H, W, Cin, dtype=x.dtype, device="cuda")
        ccv3d.ccv3d_qcache_read(desc, codes, scales, head, len(kept), back)
        assert np.array_equal(_np(back), np.stack(kept, 1))
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


def _block_reference(x, p, fmt):
    """The block on all frames x [T, H, W, C] in 64 bits: each convolution sees
    its frame as it is and the two before it as the cache gives them back."""
    T, H, W, C = x.shape

    def act_norm(v, w):
        u = norm(d(v).reshape(-1, v.shape[-1]), "rms", d(w), None, EPS)[0]
        return (u * torch.sigmoid(u)).view(v.shape)

    def conv(v, w, b):
        out = []
        held = [torch.from_numpy(quantise(_np(f), fmt)[1]).cuda() for f in v]
        wt = d(w).permute(0, 4, 1, 2, 3)
        for t in range(T):
            frames = [held[t + k - 2] if t + k - 2 >= 0 else torch.zeros_like(held[0])
                      for k in range(2)] + [d(v[t])]
            z = torch.stack(frames).permute(3, 0, 1, 2)[None]
            out.append(torch.nn.functional.conv3d(z, wt, d(b), padding=(0, 1, 1))[0, :, 0]
                       .permute(1, 2, 0))
        return torch.stack(out)

    a = conv(act_norm(x, p["n1"]), p["w1"], p["b1"])
    b = conv(act_norm(a, p["n2"]), p["w2"], p["b2"])
    return b + d(x) @ d(p["ws"]).t() + d(p["bs"])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_residual_block_streamed(fmt):
    T, H, W, C, Co = 5, 10, 18, 64, 96
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s, std=1.0, mean=0.0: (torch.randn(s, device="cuda", generator=g) * std
                                         + mean).bfloat16()
    p = dict(n1=rnd(C, mean=1.0, std=0.2), n2=rnd(Co, mean=1.0, std=0.2),
             w1=rnd(Co, 3, 3, 3, C, std=(27 * C) ** -0.5), b1=rnd(Co, std=0.1),
             w2=rnd(Co, 3, 3, 3, Co, std=(27 * Co) ** -0.5), b2=rnd(Co, std=0.1),
             ws=rnd(Co, C, std=C ** -0.5), bs=rnd(Co, std=0.1))
    x = rnd(T, H, W, C)
    px = H * W
    n1 = ccv3d.make_norm_desc(rows=px, C=C, act="silu", eps=EPS)
    n2 = ccv3d.make_norm_desc(rows=px, C=Co, act="silu", eps=EPS)
    sc = ccv3d.make_pointwise_desc(pixels=px, Cin=C, Cout=Co)
    ws = ccv3d.alloc_workspace(ccv3d.ccv3d_pointwise_workspace(sc)[0])
    q = [ccv3d.make_qcache_desc(N=1, H=H, W=W, C=c, ring_slots=3, format=fmt) for c in (C, Co)]
    rings = [ccv3d.alloc_qcache(k) for k in q]
    heads = [0, 0]
    plans = {(i, l): ccv3d.Plan(ccv3d.make_desc(N=1, Cin=c, Cout=Co, H=H, W=W, T_x=1, cache_len=l))
             for i, c in enumerate((C, Co)) for l in range(3)}
    buf = torch.empty(2 * px * Co, dtype=torch.bfloat16, device="cuda")  # shared by both modules
    y1, y2 = torch.empty(px, C, device="cuda").bfloat16(), torch.empty(px, Co, device="cuda").bfloat16()
    a, b = (torch.empty(1, 1, H, W, Co, device="cuda").bfloat16() for _ in range(2))
    out = torch.empty(T, H, W, Co, device="cuda").bfloat16()
    for t in range(T):
        l = min(t, 2)

        def conv(i, v, w, bias, o):
            c = (C, Co)[i]
            scratch = buf[:l * px * c] if l else None
            heads[i] = plans[i, l].forward_qring(v, q[i], *rings[i], heads[i], scratch, w, bias, o)

        ccv3d.ccv3d_norm_forward(n1, x[t], None, None, None, None, p["n1"], None, None, y1)
        conv(0, y1, p["w1"], p["b1"], a)
        ccv3d.ccv3d_norm_forward(n2, a, None, None, None, None, p["n2"], None, None, y2)
        conv(1, y2, p["w2"], p["b2"], b)
        ccv3d.ccv3d_pointwise_forward(sc, x[t], p["ws"], p["bs"], b, out[t], None, ws)
    torch.cuda.synchronize()
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK
    want = _block_reference(x, p, fmt)
    # five bf16 roundings in a row (two norms, two convolutions, the sum), 2^-8
    # each of values of the size of the output, and the codes that those
    # roundings flip: a flipped code of the cache is a step of 2^-6 (int8, of
    # the group's largest) or 2^-3 (e4m3, relative) in two of three taps, for
    # the share of codes within 2^-8 of a border
    step = {"int8": 2.0 ** -6, "e4m3": 2.0 ** -3}[fmt]
    err = (d(out) - want).norm() / want.norm()
    assert err <= 5 * 2.0 ** -8 + step * (2.0 ** -8 / step) ** 0.5
    m = oracle.metrics(_np(out), _np(want))
    assert m["nonfinite"] == 0


def test_block_suites_under_checked_build():
    """The bounds-checked build (libccv3d_checked.so): the suites of the operators
    around the convolution with every device address a kernel computes checked
    against its buffer.  Their far-offset tests are left to the normal build."""
    import os
    import subprocess
    import sys
    if os.environ.get("CCV3D_LIBRARY") == "checked":
        pytest.skip("already running on it")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider",
         "tests/test_gpu_norm.py", "tests/test_gpu_pointwise.py", "tests/test_gpu_qcache.py",
         "tests/test_gpu_block.py", "-k", "not far"],
        cwd=root, env=dict(os.environ, CCV3D_LIBRARY="checked"), capture_output=True, text=True,
        timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout, tail


@pytest.fixture(autouse=True)
def status_is_clean():
    """No call of a test left an error in the library's status word."""
    yield
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


def test_two_streams_at_once():
    """The operators on two streams, each with its own workspaces, overlapping on
    the GPU: the bits of the same calls one after the other."""
    def job(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
        M, C, K = 6000, 96, 192
        x, w, res, dout = rnd(M, K), rnd(C, K), rnd(M, C), rnd(M, C)
        nw, gate = rnd(C), rnd(3, C)
        nd = ccv3d.make_norm_desc(rows=M, C=C, post="rms", act="silu", gate_rows=M // 3)
        pd = ccv3d.make_pointwise_desc(pixels=M, Cin=K, Cout=C, act="silu")
        qd = ccv3d.make_qcache_desc(N=1, H=60, W=100, C=C, ring_slots=2, format="e4m3")
        ws = [ccv3d.alloc_workspace(n) for n in (ccv3d.ccv3d_norm_workspace(nd),
                                                 *ccv3d.ccv3d_pointwise_workspace(pd))]
        codes, scales = ccv3d.alloc_qcache(qd)
        out, pre, h, y, dh, db, dg, dw2, back = (torch.empty_like(t) for t in (
            res, res, res, res, res, res, gate, nw, res))
        dx, dw, dbias = torch.empty_like(x), torch.empty_like(w), torch.empty_like(nw)

        def run(stream=None):
            ccv3d.ccv3d_pointwise_forward(pd, x, w, nw, res, out, pre, ws[1], stream)
            ccv3d.ccv3d_norm_forward(nd, res, out, gate, nw, None, nw, None, h, y, stream)
            ccv3d.ccv3d_qcache_write(qd, y, 1, 0, 1, 1, codes, scales, stream)
            ccv3d.ccv3d_qcache_read(qd, codes, scales, 1, 1, back, stream)
            ccv3d.ccv3d_norm_backward(nd, h, out, gate, nw, None, nw, None, dout, res, dh, db, dg,
                                      dw2, None, None, None, ws[0], stream)
            ccv3d.ccv3d_pointwise_backward(pd, x, w, pre, db, dx, dw, dbias, ws[2], stream)
            return [out, pre, h, y, back, dh, db, dg, dw2, dx, dw, dbias]

        return run

    jobs = [job(1), job(2)]
    want = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = [j(s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("which", ["norm", "pointwise", "qcache"])
def test_first_call_of_a_process_inside_a_capture(which):
    import os
    import subprocess
    import sys
    code = """
import sys, torch
from causal_conv3d_video_b200 import ccv3d
bf = lambda *s: torch.randn(s, device="cuda").bfloat16()
if sys.argv[1] == "norm":
    h, w = bf(1000, 96), bf(96)
    out = [torch.empty_like(h), torch.empty_like(h), torch.empty_like(w)]
    d = ccv3d.make_norm_desc(rows=1000, C=96, act="silu")
    ws = ccv3d.alloc_workspace(ccv3d.ccv3d_norm_workspace(d))
    def call():
        ccv3d.ccv3d_norm_forward(d, h, None, None, None, None, w, None, None, out[0])
        ccv3d.ccv3d_norm_backward(d, h, None, None, None, None, w, None, h, None, out[1], None,
                                  None, None, None, out[2], None, ws)
elif sys.argv[1] == "pointwise":
    x, w = bf(1000, 192), bf(96, 192)
    out = [bf(1000, 96), torch.empty_like(x), torch.empty_like(w)]
    d = ccv3d.make_pointwise_desc(pixels=1000, Cin=192, Cout=96)
    ws = [ccv3d.alloc_workspace(n) for n in ccv3d.ccv3d_pointwise_workspace(d)]
    def call():
        ccv3d.ccv3d_pointwise_forward(d, x, w, None, None, out[0], None, ws[0])
        ccv3d.ccv3d_pointwise_backward(d, x, w, None, out[0], out[1], out[2], None, ws[1])
else:
    x = bf(1, 1, 8, 8, 96)
    d = ccv3d.make_qcache_desc(N=1, H=8, W=8, C=96, ring_slots=2)
    out = [torch.empty_like(x), *ccv3d.alloc_qcache(d)]
    def call():
        ccv3d.ccv3d_qcache_write(d, x, 1, 0, 1, 1, out[1], out[2])
        ccv3d.ccv3d_qcache_read(d, out[1], out[2], 1, 1, out[0])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, out))
assert ccv3d.ccv3d_block_get_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code, which], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def _qring_against_dense(conv, env, fmt, chunks, extra=0, check_oracle=True):
    """forward_qring chunk by chunk against the same plan's forward on the frames
    that the ring gives back: the same bits, whatever kernel convolves."""
    g = torch.Generator(device="cuda").manual_seed(9)
    dt = torch.bfloat16 if conv.dtype == "bf16" else torch.float32
    rnd = lambda *s, std=1.0: (torch.randn(s, device="cuda", generator=g) * std).to(dt)
    w = rnd(conv.Cout, conv.kt, conv.kh, conv.kw, conv.Cin,
            std=(conv.kt * conv.kh * conv.kw * conv.Cin) ** -0.5)
    b = rnd(conv.Cout, std=0.1) if conv.has_bias else None
    slots = conv.cache_keep + min(conv.cache_keep, conv.T_x) + extra
    desc = ccv3d.make_qcache_desc(N=conv.N, H=conv.H, W=conv.W, C=conv.Cin, ring_slots=slots,
                                  format=fmt, dtype=conv.dtype)
    codes, scales = ccv3d.alloc_qcache(desc)
    head, length = slots - 1, 0
    for _ in range(chunks):
        c = conv.replace(cache_len=length)
        with plan_env(env):
            plan = ccv3d.Plan(ccv3d.desc_for(c))
        x = rnd(c.N, c.T_x, c.H, c.W, c.Cin)
        cache = torch.empty(c.N, length, c.H, c.W, c.Cin, dtype=dt, device="cuda") if length else None
        if length:
            ccv3d.ccv3d_qcache_read(desc, codes, scales, head, length, cache)
        want, nc = plan.alloc_outputs("cuda")
        plan.forward(x, cache, w, b, want, nc)
        out, _ = plan.alloc_outputs("cuda")
        out.fill_(float("nan"))
        buf = torch.full_like(cache, float("nan")) if length else None
        before = codes.clone()
        new_head = plan.forward_qring(x, desc, codes, scales, head, buf, w, b, out)
        torch.cuda.synchronize()
        assert plan.status() == ccv3d.CCV3D_OK
        assert torch.equal(out, want), (c.name, plan.kernel, length)
        assert buf is None or torch.equal(buf, cache)
        writes, keep = plan.ring_writes(), plan.sizes["new_cache_frames"]
        assert new_head == (head + length + writes - keep) % slots
        fresh = torch.zeros_like(codes)
        ccv3d.ccv3d_qcache_write(desc, x, c.T_x, c.T_x - writes, writes, (head + length) % slots,
                                 fresh, scales.clone())
        at = [(head + length + i) % slots for i in range(writes)]
        shape = (c.N, slots, -1)
        for s in range(slots):
            ref = fresh if s in at else before
            assert torch.equal(codes.view(shape)[:, s], ref.view(shape)[:, s]), (c.name, s)
        if check_oracle:
            ref, _ = oracle.forward(oracle_params(c), _np(x), _np(cache) if length else None, _np(w),
                                    _np(b) if b is not None else None)
            assert_close(_np(out), ref, c.dtype, c.name)
        head, length = new_head, keep


@pytest.mark.parametrize("fmt", ["int8", "e2m1"])
@pytest.mark.parametrize("conv,env", RING_SIGS, ids=lambda v: getattr(v, "name", None) or "env")
def test_forward_qring_every_kernel(conv, env, fmt):
    _qring_against_dense(conv, env, fmt, 4, extra=1)


@pytest.mark.parametrize("conv", [
    Conv("q384_90x160", 384, 384, 90, 160, T_x=1, cache_len=0),
    Conv("q192_360x640_t2", 192, 192, 360, 640, T_x=2, cache_len=0),
    Conv("q96_720x1280_t4", 96, 96, 720, 1280, T_x=4, cache_len=0),
    Conv("q96to3_720x1280_t4", 96, 3, 720, 1280, T_x=4, cache_len=0),
], ids=lambda c: c.name)
def test_forward_qring_decoder_sizes(conv):
    """The kernels that the planner picks at the decoder's own sizes."""
    _qring_against_dense(conv, {}, "e4m3", 3, check_oracle=False)


def _poison(tensors):
    for t in tensors:
        t.fill_(255 if t.dtype == torch.uint8 else float("nan"))


def test_two_streams_overlapping_from_poison():
    """Two jobs of all the operators, each captured three times in a row, replayed
    at once on two streams from poisoned outputs, workspaces and rings: after each
    round the bits of the jobs run one after the other, and the replays did
    overlap."""
    def job(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
        M, C, K = 24000, 96, 192
        x, w, res, dout = rnd(M, K), rnd(C, K), rnd(M, C), rnd(M, C)
        nw, gate = rnd(C), rnd(3, C)
        nd = ccv3d.make_norm_desc(rows=M, C=C, post="rms", act="silu", gate_rows=M // 3)
        pd = ccv3d.make_pointwise_desc(pixels=M, Cin=K, Cout=C, act="silu")
        few = ccv3d.make_pointwise_desc(pixels=5, Cin=K, Cout=C)
        qd = ccv3d.make_qcache_desc(N=1, H=120, W=200, C=C, ring_slots=2, format="e4m3")
        ws = [ccv3d.alloc_workspace(n) for n in (ccv3d.ccv3d_norm_workspace(nd),
                                                 *ccv3d.ccv3d_pointwise_workspace(pd))]
        codes, scales = ccv3d.alloc_qcache(qd)
        out, pre, h, y, dh, db, dg, dw2, back = (torch.empty_like(t) for t in (
            res, res, res, res, res, res, gate, nw, res))
        dx, dw, dbias = torch.empty_like(x), torch.empty_like(w), torch.empty_like(nw)
        rows = torch.empty(5, C, device="cuda").bfloat16()
        written = [out, pre, h, y, back, dh, db, dg, dw2, dx, dw, dbias, rows]

        def run():
            ccv3d.ccv3d_pointwise_forward(pd, x, w, nw, res, out, pre, ws[1])
            ccv3d.ccv3d_norm_forward(nd, res, out, gate, nw, None, nw, None, h, y)
            ccv3d.ccv3d_qcache_write(qd, y, 1, 0, 1, 1, codes, scales)
            ccv3d.ccv3d_qcache_read(qd, codes, scales, 1, 1, back)
            ccv3d.ccv3d_norm_backward(nd, h, out, gate, nw, None, nw, None, dout, res, dh, db, dg,
                                      dw2, None, None, None, ws[0])
            ccv3d.ccv3d_pointwise_backward(pd, x, w, pre, db, dx, dw, dbias, ws[2])
            ccv3d.ccv3d_pointwise_forward(few, dx[:5], w, None, None, rows, None, None)

        return run, written, [t for t in (*ws, codes, scales) if t is not None]

    jobs = [job(1), job(2)]
    want = []
    for run, written, scratch in jobs:
        _poison(written + scratch)
        run()
        torch.cuda.synchronize()
        assert all(t.isfinite().all() for t in written)
        want.append([t.clone() for t in written])
    graphs, streams = [], [torch.cuda.Stream() for _ in jobs]
    for (run, _, _), st in zip(jobs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                run()
        graphs.append(g)
    overlapped = False
    for _ in range(10):
        for _, written, scratch in jobs:
            _poison(written + scratch)
        torch.cuda.synchronize()
        ev = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in jobs]
        for g, st, (a, b) in zip(graphs, streams, ev):
            with torch.cuda.stream(st):
                a.record()
                g.replay()
                b.record()
        torch.cuda.synchronize()
        for (_, written, _), ref in zip(jobs, want):
            assert all(torch.equal(t, r) for t, r in zip(written, ref))
        # the second began before the first ended, and ended after it began
        overlapped |= ev[1][0].elapsed_time(ev[0][1]) > 0 and ev[0][0].elapsed_time(ev[1][1]) > 0
    assert overlapped


@pytest.mark.parametrize("which", ["norm", "pointwise", "few", "qcache"])
def test_first_call_inside_a_capture_computes(which):
    """As above from poisoned outputs, the replay and an eager call each against
    the definition in 64 bits."""
    import os
    import subprocess
    import sys
    code = """
import sys, torch
sys.path[:0] = ["tests"]
from block_util import HALF, ROW, act, close, d, norm
from causal_conv3d_video_b200 import ccv3d
gen = torch.Generator(device="cuda").manual_seed(1)
bf = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()
half = HALF["bf16"]
acc = lambda k: (k + 16) * 2.0 ** -23
if sys.argv[1] == "norm":
    h, w = bf(1000, 96), bf(96)
    out = [torch.empty_like(h), torch.empty_like(h), torch.empty_like(w)]
    nd = ccv3d.make_norm_desc(rows=1000, C=96)
    ws = ccv3d.alloc_workspace(ccv3d.ccv3d_norm_workspace(nd))
    def call():
        ccv3d.ccv3d_norm_forward(nd, h, None, None, None, None, w, None, None, out[0])
        ccv3d.ccv3d_norm_backward(nd, h, None, None, None, None, w, None, h, None, out[1], None,
                                  None, None, None, out[2], None, ws)
    def check():
        y, n, rstd, mag = norm(d(h), "rms", d(w), None, 1e-6)
        close(out[0], y, half * y.abs() + ROW["bf16"] * mag, "y")
        dn = d(h) * d(w)
        dh = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
        m = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
        close(out[1], dh, half * dh.abs() + 4 * ROW["bf16"] * m, "dh")
        t = d(h) * n
        close(out[2], t.sum(0), half * t.sum(0).abs() + 4 * ROW["bf16"] * t.abs().sum(0), "dw")
elif sys.argv[1] in ("pointwise", "few"):
    M = 1000 if sys.argv[1] == "pointwise" else 5
    x, w, g = bf(M, 192), bf(96, 192), bf(M, 96)
    out = [bf(M, 96), torch.empty_like(x), torch.empty_like(w)]
    pd = ccv3d.make_pointwise_desc(pixels=M, Cin=192, Cout=96)
    ws = [ccv3d.alloc_workspace(n) for n in ccv3d.ccv3d_pointwise_workspace(pd)]
    def call():
        ccv3d.ccv3d_pointwise_forward(pd, x, w, None, None, out[0], None, ws[0])
        ccv3d.ccv3d_pointwise_backward(pd, x, w, None, g, out[1], out[2], None, ws[1])
    def check():
        for got, a, b, k in ((out[0], d(x), d(w).t(), 192), (out[1], d(g), d(w), 96),
                             (out[2], d(g).t(), d(x), M)):
            want = a @ b
            close(got, want, half * want.abs() + acc(k) * (a.abs() @ b.abs()), "product")
else:
    # integers with a 127 in each group of 32: scale 1, read back as they are
    x = torch.randint(-127, 128, (1, 1, 8, 8, 96), device="cuda", generator=gen).bfloat16()
    x[..., ::32] = 127
    qd = ccv3d.make_qcache_desc(N=1, H=8, W=8, C=96, ring_slots=2)
    out = [torch.empty_like(x), *ccv3d.alloc_qcache(qd)]
    def call():
        ccv3d.ccv3d_qcache_write(qd, x, 1, 0, 1, 1, out[1], out[2])
        ccv3d.ccv3d_qcache_read(qd, out[1], out[2], 1, 1, out[0])
    def check():
        assert torch.equal(out[0], x)
        assert (out[2].view(2, -1)[1] == 127).all() and (out[2].view(2, -1)[0] == 255).all()
def poison():
    for t in out:
        t.fill_(255 if t.dtype == torch.uint8 else float("nan"))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
poison()
graph.replay()
torch.cuda.synchronize()
check()
got = [t.clone() for t in out]
poison()
call()
torch.cuda.synchronize()
check()
assert all(torch.equal(a, b) for a, b in zip(got, out))
assert ccv3d.ccv3d_block_get_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code, which], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_forward_qring_with_a_larger_scratch():
    """cache_buf may be larger than the call's frames: only those are written."""
    H, W, C = 6, 10, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
    x, w, b = rnd(1, 1, H, W, C), rnd(C, 3, 3, 3, C), rnd(C)
    q = ccv3d.make_qcache_desc(N=1, H=H, W=W, C=C, ring_slots=3)
    plan = ccv3d.Plan(ccv3d.make_desc(N=1, Cin=C, Cout=C, H=H, W=W, T_x=1, cache_len=2))
    outs = []
    for frames in (2, 5):
        codes, scales = ccv3d.alloc_qcache(q)
        ccv3d.ccv3d_qcache_write(q, rnd(1, 2, H, W, C) if not outs else held, 2, 0, 2, 0, codes, scales)
        if not outs:
            held = torch.empty(1, 2, H, W, C, device="cuda").bfloat16()
            ccv3d.ccv3d_qcache_read(q, codes, scales, 0, 2, held)
        buf = torch.full((1, frames, H, W, C), 7.0, device="cuda").bfloat16()
        out, _ = plan.alloc_outputs("cuda")
        assert plan.forward_qring(x, q, codes, scales, 0, buf, w, b, out) == 1
        outs.append(out)
        assert torch.equal(buf[:, :2], held) and (buf[:, 2:] == 7.0).all()
    assert torch.equal(*outs)
