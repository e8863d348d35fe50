"""The ring cache in 8 and 4 bits: every code, scale and value read back is
equal to the definition's, computed in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

from causal_conv3d_video_b200 import ccv3d

pytestmark = pytest.mark.gpu

E4M3 = np.array([i * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10)
                 for i in range(127)])
GRID = {"int8": np.arange(128.0), "e4m3": E4M3, "e2m1": np.array([0, .5, 1, 1.5, 2, 3, 4, 6])}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def quantise(x, fmt):
    """(scale bytes [..., groups], codes as indexes into GRID with sign, values)
    of x [..., C], by search for the nearest value, ties to the even index."""
    grid = GRID[fmt]
    C = x.shape[-1]
    scales = np.zeros(x.shape[:-1] + (-(-C // 32),), np.uint8)
    values = np.zeros_like(x)
    for g in range(scales.shape[-1]):
        v = x[..., 32 * g:32 * g + 32]
        most = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
        e = np.full(most.shape, -126)
        for t in range(-126, 128):   # the smallest exponent that fits
            e = np.where(grid[-1] * 2.0 ** e.astype(float) < np.where(bad, 0, most), t, e)
        scales[..., g] = np.where(bad, 255, e + 127)
        step = 2.0 ** e.astype(float)[..., None]
        a = np.where(np.isfinite(v), np.abs(v), 0) / step
        hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
        lo = hi - 1
        dl, dh = a - grid[lo], grid[hi] - a
        idx = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
        values[..., 32 * g:32 * g + 32] = np.where(bad[..., None], np.nan,
                                                   np.sign(v) * grid[idx] * step)
    return scales, values


def unpack(codes, C, fmt):
    """Values of the code bytes, before their scale."""
    c = codes.astype(np.int64)
    if fmt == "int8":
        return codes.view(np.int8).astype(float)
    if fmt == "e2m1":
        c = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))[..., :C]
        return np.where(c >= 8, -1, 1) * GRID[fmt][c % 8]
    return np.where(c >= 128, -1, 1) * GRID[fmt][np.minimum(c % 128, 126)]


def _values(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[-1], generator=g))
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    # ties, borders of the formats, tiny and huge values, zeros
    flat[0] = 0
    flat[n // 3] = torch.arange(shape[-1]) % 13 * 0.25 - 1.5
    flat[n // 2] *= 2.0 ** -125
    flat[n - 1] *= 2.0 ** 100
    flat[n // 4, 0] = 448.0
    flat[n // 5, -1] = 127.0
    flat[n // 6, 0] = 6.0
    return x.to(DT[dtype])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,W,C,slots", [
    (1, 9, 11, 96, 3), (2, 5, 7, 16, 4), (1, 3, 5, 33, 3), (1, 13, 1, 1, 2), (2, 4, 6, 100, 5),
    (1, 6, 5, 40, 3), (1, 2, 3, 1055, 3), (1, 1, 1, 2048, 1), (1, 8, 9, 64, 2), (3, 4, 4, 31, 4),
    (1, 7, 5, 68, 3), (2, 5, 3, 12, 3), (1, 9, 4, 202, 2), (1, 33, 40, 6, 2)])
def test_write_and_read_exact(N, H, W, C, slots, dtype, fmt):
    desc = ccv3d.make_qcache_desc(N=N, H=H, W=W, C=C, ring_slots=slots, format=fmt, dtype=dtype)
    cb, sb = ccv3d.ccv3d_qcache_sizes(desc)
    pad = 64
    codes_buf = torch.full((cb + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    scales_buf = torch.full((sb + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    codes, scales = codes_buf[pad:pad + cb], scales_buf[pad:pad + sb]
    T = slots + 1
    frames = max(1, slots - 1)
    for slot, first in [(0, 0), (slots - 1, T - frames)]:
        x = _values((N, T, H, W, C), dtype, 3 * slot + 1)
        codes.fill_(0x5A)
        scales.fill_(0x5A)
        ccv3d.ccv3d_qcache_write(desc, x.cuda(), T, first, frames, slot, codes, scales)
        back = torch.full((N, frames, H, W, C), 7.0, dtype=DT[dtype], device="cuda")
        ccv3d.ccv3d_qcache_read(desc, codes, scales, slot, frames, back)
        torch.cuda.synchronize()
        want_s, want_v = quantise(x[:, first:first + frames].double().numpy(), fmt)
        at = [(slot + i) % slots for i in range(frames)]
        cbytes = cb // (N * slots * H * W)
        got_c = codes.cpu().numpy().reshape(N, slots, H, W, cbytes)
        got_s = scales.cpu().numpy().reshape(N, slots, H, W, -1)
        assert np.array_equal(got_s[:, at], want_s)
        step = np.repeat(2.0 ** (want_s.astype(float) - 127), 32, -1)[..., :C]
        assert np.array_equal(unpack(got_c[:, at], C, fmt) * step, want_v)
        # what is read back is the code's value, rounded once to the type
        want_t = torch.from_numpy(want_v).to(DT[dtype])
        assert torch.equal(back.cpu(), want_t)
        rest = [i for i in range(slots) if i not in at]
        assert (got_c[:, rest] == 0x5A).all() and (got_s[:, rest] == 0x5A).all()
    for buf, n in ((codes_buf, cb), (scales_buf, sb)):
        assert (buf[:pad] == 0x5A).all() and (buf[pad + n:] == 0x5A).all()
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e2m1"])
def test_every_bf16_value(fmt):
    """Each of the 65536 bf16 values as its group's largest and next to one."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(1 << 16, 32, dtype=torch.bfloat16)
    x[:, 0] = bits
    x[:, 1] = bits / 3
    x[:, 2] = bits * 0.30078125
    x[:, 31] = -bits / 2
    desc = ccv3d.make_qcache_desc(N=1, H=256, W=256, C=32, ring_slots=1, format=fmt)
    codes, scales = ccv3d.alloc_qcache(desc)
    back = torch.empty(1, 1, 256, 256, 32, dtype=torch.bfloat16, device="cuda")
    ccv3d.ccv3d_qcache_write(desc, x.cuda(), 1, 0, 1, 0, codes, scales)
    ccv3d.ccv3d_qcache_read(desc, codes, scales, 0, 1, back)
    torch.cuda.synchronize()
    want_s, want_v = quantise(x.double().numpy(), fmt)
    assert np.array_equal(scales.cpu().numpy().reshape(-1, 1), want_s)
    want = torch.from_numpy(want_v).to(torch.bfloat16)
    got = back.cpu().view(-1, 32)
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want[~nan])
    # a NaN or an infinity takes its own group and no other
    assert (scales.cpu().view(-1) == 255).sum() == int((~x.float().isfinite()).any(1).sum())


def test_every_code_reads_back():
    """All 256 scale bytes with all code bytes, also those no write produces."""
    for fmt, dtype in itertools.product(["int8", "e4m3", "e2m1"], ["bf16", "fp32"]):
        C = 64 if fmt == "e2m1" else 32
        n = 256 * 8
        desc = ccv3d.make_qcache_desc(N=1, H=n, W=1, C=C, ring_slots=1, format=fmt, dtype=dtype)
        codes = torch.arange(256, dtype=torch.uint8).view(8, 32).repeat(256, 1).cuda()
        per = 2 if fmt == "e2m1" else 1
        scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(8 * per).cuda()
        out = torch.empty(1, 1, n, 1, C, dtype=DT[dtype], device="cuda")
        ccv3d.ccv3d_qcache_read(desc, codes, scales, 0, 1, out)
        c = codes.cpu().numpy()
        v = unpack(c, C, fmt)
        if fmt == "e4m3":
            v = np.where(c % 128 == 127, np.nan, v)
        s = scales.cpu().numpy().reshape(n, per).astype(float)
        want = np.repeat(np.where(s == 255, np.nan, 2.0 ** (s - 127)), 32, -1) * v
        want_t = torch.from_numpy(want).float().to(DT[dtype])
        got = out.cpu().view(n, C)
        assert torch.equal(got.isnan(), want_t.isnan())
        ok = ~want_t.isnan()
        assert torch.equal(got[ok], want_t[ok]), (fmt, dtype)


def test_far_frames():
    """Slots past 2^32 bytes of a large ring."""
    H, W, C, slots = 720, 1280, 96, 52
    desc = ccv3d.make_qcache_desc(N=1, H=H, W=W, C=C, ring_slots=slots, format="int8")
    codes, scales = ccv3d.alloc_qcache(desc)
    x = torch.randn(1, 1, H, W, C, device="cuda").bfloat16()
    ccv3d.ccv3d_qcache_write(desc, x, 1, 0, 1, slots - 1, codes, scales)
    small = ccv3d.make_qcache_desc(N=1, H=H, W=W, C=C, ring_slots=1, format="int8")
    c2, s2 = ccv3d.alloc_qcache(small)
    ccv3d.ccv3d_qcache_write(small, x, 1, 0, 1, 0, c2, s2)
    assert torch.equal(codes.view(slots, -1)[-1], c2) and torch.equal(scales.view(slots, -1)[-1], s2)
    assert int(codes.view(slots, -1)[:-1].any()) == 0
    a, b = torch.empty_like(x), torch.empty_like(x)
    ccv3d.ccv3d_qcache_read(desc, codes, scales, slots - 1, 1, a)
    ccv3d.ccv3d_qcache_read(small, c2, s2, 0, 1, b)
    assert torch.equal(a, b)


def test_graph_and_stream():
    desc = ccv3d.make_qcache_desc(N=1, H=16, W=20, C=96, ring_slots=3, format="e2m1")
    codes, scales = ccv3d.alloc_qcache(desc)
    x = torch.randn(1, 1, 16, 20, 96, device="cuda").bfloat16()
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccv3d.ccv3d_qcache_write(desc, x, 1, 0, 1, 2, codes, scales)
        ccv3d.ccv3d_qcache_read(desc, codes, scales, 2, 1, out)
    for seed in range(2):
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        _, want = quantise(x.double().cpu().numpy(), "e2m1")
        assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.fixture(autouse=True)
def status_is_clean():
    """No call of a test left an error (a wait that ran out; in the checked build
    an address outside its buffer) in the library's status word."""
    yield
    assert ccv3d.ccv3d_block_get_status() == ccv3d.CCV3D_OK
