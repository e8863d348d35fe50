"""The bounded waits of the operators around the convolution: where one runs out,
the kernel records it, asks for no more copies, waits for those in flight and
stores nothing of what it did not get; the context stays usable.  The kernels
are compiled here with a short limit and one bulk copy left out
(tests/c/block_waits.cu): nothing faults and every wait ends."""
import ctypes
import os
import subprocess

import pytest
import torch

from block_util import HALF, ROW, close, d, norm
from causal_conv3d_video_b200 import build

pytestmark = pytest.mark.gpu

C, EPS = 96, 1e-6
TIMEOUT = 7
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("waits") / "block_waits.so")
    subprocess.check_call([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler",
                           "-fPIC,-fvisibility=hidden", "-I", os.path.join(build.ROOT, "include"),
                           "-I", build.CSRC,
                           os.path.join(HERE, "c", "block_waits.cu"), "-o", so])
    lib = ctypes.CDLL(so)
    p, ll, i, ip = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.tile_shape.argtypes = [i, ll, ip, ip]
    lib.norm_forward.argtypes = [p] * 4 + [ll, i, ip]
    lib.norm_backward.argtypes = [p] * 7 + [ll, i, ip]
    lib.few_rows_product.argtypes = [p] * 3 + [i, i, i, ip]
    return lib


def _bf(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).bfloat16()


def _like(t):
    return torch.full_like(t, 7.0)


def _call(f, *args):
    torch.cuda.synchronize()
    issued = ctypes.c_int()
    status = f(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args],
               ctypes.byref(issued))
    return status, issued.value


def _tiles(lib, backward, rows):
    """Rows of a tile, tiles, stages of the ring."""
    per, stages = ctypes.c_int(), ctypes.c_int()
    lib.tile_shape(backward, rows, ctypes.byref(per), ctypes.byref(stages))
    return per.value, -(-rows // per.value), stages.value


@pytest.mark.parametrize("tile", [0, 1, 5, 19])
def test_norm_forward_wait_runs_out(waits, tile):
    rows = 1270
    per, tiles, stages = _tiles(waits, 0, rows)
    tile = min(tile, tiles - 1)
    h, b = _bf(rows, C), _bf(rows, C, seed=1)
    whole = _like(h), _like(h)
    status, issued = _call(waits.norm_forward, h, b, *whole, rows, -1)
    assert (status, issued) == (0, 2 * tiles)
    p, _, _, mag = norm(d(b), "rms", None, None, EPS)
    want = d(h) + p
    close(whole[0], want, HALF["bf16"] * want.abs() + ROW["bf16"] * (d(h).abs() + mag), "h_out")
    part = _like(h), _like(h)
    status, issued = _call(waits.norm_forward, h, b, *part, rows, 2 * tile + 1)
    assert status == TIMEOUT
    assert issued == 2 * min(tile + stages, tiles)
    for got, all_of_it in zip(part, whole):
        assert torch.equal(got[:tile * per], all_of_it[:tile * per])
        assert (got[tile * per:] == 7.0).all()


@pytest.mark.parametrize("tile", [0, 2, 11])
def test_norm_backward_wait_runs_out(waits, tile):
    rows = 760
    per, tiles, stages = _tiles(waits, 1, rows)
    tile = min(tile, tiles - 1)
    ins = [_bf(rows, C, seed=i) for i in range(4)]
    part = torch.full((2, C), 7.0, device="cuda")
    whole = _like(ins[0]), _like(ins[0])
    status, issued = _call(waits.norm_backward, *ins, *whole, part, rows, -1)
    assert (status, issued) == (0, 4 * tiles)
    # the column sum of du n: 2^-24 of the terms' magnitudes a dependent addition, of
    # which a thread has rows / 64 and the block a few more
    n = norm(d(ins[0]), "rms", None, None, EPS)[1]
    terms = d(ins[2]) * n
    close(part[0], terms.sum(0), (rows // 64 + 64) * 2.0 ** -24 * terms.abs().sum(0), "sum du n")
    part.fill_(7.0)
    got = _like(ins[0]), _like(ins[0])
    status, issued = _call(waits.norm_backward, *ins, *got, part, rows, 4 * tile + 2)
    assert status == TIMEOUT
    assert issued == 4 * min(tile + stages, tiles)
    assert (part == 7.0).all()
    for g, w in zip(got, whole):
        assert torch.equal(g[:tile * per], w[:tile * per])
        assert (g[tile * per:] == 7.0).all()


@pytest.mark.parametrize("chunk", [0, 2, 5, 6, 7])
def test_few_rows_product_wait_runs_out(waits, chunk):
    M, chunks = 5, 8
    K = 512 * chunks - 264
    x, w = _bf(M, K), _bf(8, K, seed=1)
    out = torch.full((M, 8), 7.0, device="cuda", dtype=torch.bfloat16)
    status, issued = _call(waits.few_rows_product, x, w, out, M, K, -1)
    assert (status, issued) == (0, 8 * chunks)
    want, mag = d(x) @ d(w).t(), d(x).abs() @ d(w).abs().t()
    close(out, want, HALF["bf16"] * want.abs() + (K + 16) * 2.0 ** -23 * mag, "out")
    out.fill_(7.0)
    status, issued = _call(waits.few_rows_product, x, w, out, M, K, 8 * chunk + 3)
    assert status == TIMEOUT
    assert issued == 8 * min(chunk + 3, chunks)
    assert (out == 7.0).all()
