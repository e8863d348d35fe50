"""The range checks of the operators around the convolution, in kernels compiled
as the bounds-checked build does (tests/c/block_ranges.cu) and launched with
more blocks or gate rows than their parameters allow for: the violation is
recorded and nothing outside the buffers that the parameters describe is
written.  The allocations reach further than that, so no access is out of range
in memory."""
import ctypes
import os
import subprocess

import pytest
import torch

from causal_conv3d_video_b200 import build

pytestmark = pytest.mark.gpu

BOUNDS = 9
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ranges(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ranges") / "block_ranges.so")
    subprocess.check_call([build._nvcc(), *build.ARCH, "-DCCV3D_CHECKED", "-O1", "-std=c++17",
                           "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                           "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC,
                           os.path.join(HERE, "c", "block_ranges.cu"), "-o", so])
    lib = ctypes.CDLL(so)
    p, ll, i = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int
    lib.cache_write.argtypes = lib.cache_read.argtypes = [p] * 3 + [i] * 6
    lib.norm_forward.argtypes = [p] * 5 + [i, ll, ll]
    lib.norm_backward.argtypes = [p] * 8 + [i, ll, i]
    return lib


def _bf(*shape):
    g = torch.Generator(device="cuda").manual_seed(3)
    return torch.randn(shape, device="cuda", generator=g).bfloat16()


def _call(f, *args):
    torch.cuda.synchronize()
    return f(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args])


@pytest.mark.parametrize("C", [96, 40, 33])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_cache_past_its_entries(ranges, C, fmt):
    px, slots, frames = 70, 3, 2
    x = _bf(2, frames, px, C)
    cb, sb = (C + 1) // 2 if fmt == 2 else C, (C + 31) // 32
    codes = torch.full((2, slots, px, cb), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, slots, px, sb), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((2, frames, px, C), 7.0, dtype=torch.bfloat16, device="cuda")
    assert _call(ranges.cache_write, x, codes, scales, C, fmt, px, slots, frames, 1) == 0
    assert (scales[0, :frames] != 0x5A).any() and (codes[0, :frames] != 0x5A).any()
    assert _call(ranges.cache_read, out, codes, scales, C, fmt, px, slots, frames, 1) == 0
    assert (out[0] != 7.0).any() and (out[1] == 7.0).all()
    assert _call(ranges.cache_write, x, codes, scales, C, fmt, px, slots, frames, 2) == BOUNDS
    assert (codes[1] == 0x5A).all() and (scales[1] == 0x5A).all()
    assert _call(ranges.cache_read, out, codes, scales, C, fmt, px, slots, frames, 2) == BOUNDS
    assert (out[1] == 7.0).all()


@pytest.mark.parametrize("C", [96, 1024])
def test_norm_forward_past_its_gates(ranges, C):
    rows = 500
    h, b, gate = _bf(rows, C), _bf(rows, C), _bf(2, C)
    h_out, y = torch.empty_like(h), torch.empty_like(h)
    assert _call(ranges.norm_forward, h, b, gate, h_out, y, C, rows, 250) == 0
    # 500 rows in groups of 300: one whole group, and rows of a second
    assert _call(ranges.norm_forward, h, b, gate, h_out, y, C, rows, 300) == BOUNDS


@pytest.mark.parametrize("C", [96, 1024])
def test_norm_backward_past_its_groups(ranges, C):
    rows = 200
    ins = [_bf(2 * rows, C), _bf(2 * rows, C), _bf(2, C), _bf(2 * rows, C), _bf(2 * rows, C)]
    dh, db = (torch.full((2 * rows, C), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    part = torch.full((2, 2, C), 7.0, device="cuda")

    def call(groups):
        return _call(ranges.norm_backward, *ins, dh, db, part, C, rows, groups)

    assert call(1) == 0
    assert (dh[:rows] != 7.0).any() and (db[:rows] != 7.0).any() and (part[0] != 7.0).any()
    assert (dh[rows:] == 7.0).all() and (part[1] == 7.0).all()
    assert call(2) == BOUNDS
    assert (dh[rows:] == 7.0).all() and (db[rows:] == 7.0).all()
