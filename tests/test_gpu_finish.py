"""The kernels that add the parts of a product (mid_finish_kernel, dense_finish_kernel) where a part is
missing: a CTA whose wait ran out marks its parts, and outputs that need one stay as they were. No wait is made
to run out here: the parts, and the marks among them, are written by the test.

The other outputs are exact: the parts are added in order in fp32, which numpy repeats, and rounded once."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from calibration_free_weight_hqq_b200 import build

pytestmark = pytest.mark.gpu

BEFORE = 7.0


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("native") / "libfinish.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "finish_kernels.cu")
    flags = [f for f in build.NVCC_FLAGS if f not in ("-Xptxas", "-v")]
    subprocess.check_call([build.nvcc(), *flags, "-I" + build.CSRC, "-shared", src, "-o", out])
    L = ctypes.CDLL(out)
    L.no_part.restype = ctypes.c_uint
    P, I = ctypes.c_void_p, ctypes.c_int
    L.mid_finish.argtypes = [P] * 4 + [I] * 8
    L.dense_finish.argtypes = [P] * 4 + [I] * 4
    return L


def on_device(parts, mark):
    """The parts, with NaN in place of the marks turned into them."""
    bits = parts.view(np.uint32).copy()
    bits[np.isnan(parts)] = mark
    return torch.from_numpy(bits.view(np.int32)).cuda()


def outputs(shape, n):
    return [torch.full(shape, BEFORE, dtype=torch.bfloat16, device="cuda") for _ in range(n)]


def check(got, sums, missing):
    """got: Y alone, or Y, G and U; sums: fp32, one or two."""
    keep = torch.from_numpy(~missing).cuda()
    want = [torch.from_numpy(s).cuda().bfloat16() for s in sums]
    for g, w in zip(got[1:] or got, want):
        assert torch.equal(torch.where(keep, g, BEFORE), torch.where(keep, w, BEFORE))
    for g in got:
        assert (g[~keep] == BEFORE).all()
    if len(got) == 3:  # Y = silu(g) u of the unrounded sums, within 2^-8 and the special function's 2^-18
        g, u = (torch.from_numpy(s).cuda().double() for s in sums)
        y = g * torch.sigmoid(g) * u
        assert ((got[0].double() - y).abs() <= 2.0 ** -8 * (1 + 2.0 ** -9) * y.abs() + 1e-30)[keep].all()


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,out,tok_tiles,row_tiles,kb,ctas", [(13, 200, 1, 2, 5, 4), (40, 520, 2, 5, 7, 19),
                                                             (30, 128, 1, 1, 9, 4), (48, 384, 3, 3, 4, 7)])
def test_tiles_with_a_missing_part(kernels, mats, M, out, tok_tiles, row_tiles, kb, ctas):
    tok = ((M + tok_tiles - 1) // tok_tiles + 15) // 16 * 16
    rng = np.random.default_rng(M)
    parts = rng.standard_normal((ctas, 2, mats, tok, 128)).astype(np.float32)
    units = row_tiles * tok_tiles * kb
    first = [c * units // ctas for c in range(ctas + 1)]
    lost = rng.choice(ctas, max(1, ctas // 4), replace=False)
    sums = np.zeros((mats, tok_tiles * tok, row_tiles * 128), np.float32)
    missing = np.ones(sums.shape[1:], bool)  # a tile that one CTA has alone is not this kernel's
    shared = 0
    for tile in range(row_tiles * tok_tiles):
        owners = [c for c in range(ctas) if first[c] < (tile + 1) * kb and first[c + 1] > tile * kb]
        if len(owners) == 1:
            continue
        shared += 1
        slots = [(c, 0 if first[c] // kb == tile else 1) for c in owners]
        for c, s in slots:
            if c in lost:
                parts[c, s, 0] = np.nan
        total = parts[slots[0]].copy()
        for s in slots[1:]:
            total = total + parts[s]
        at = np.s_[tile % tok_tiles * tok:(tile % tok_tiles + 1) * tok,
                   tile // tok_tiles * 128:(tile // tok_tiles + 1) * 128]
        sums[(slice(None),) + at] = total
        missing[at] = any(c in lost for c in owners)
    assert shared and missing.any() and (not missing.all() or shared == 1)
    Y = outputs((M, out), 1 if mats == 1 else 3)
    p = on_device(parts, kernels.no_part())
    assert kernels.mid_finish(p.data_ptr(), *[t.data_ptr() for t in Y], *[None] * (3 - len(Y)), M, out, tok,
                              tok_tiles, row_tiles, kb, ctas, mats) == 0
    # tokens of the last tile past M do not exist
    check(Y, np.ascontiguousarray(sums[:, :M, :out]), missing[:M, :out])


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("M,N,splits", [(1, 8, 2), (130, 264, 4), (70, 1032, 3)])
def test_sums_with_a_missing_part(kernels, kind, M, N, splits):
    mats = 2 if kind == 1 else 1
    rng = np.random.default_rng(M + kind)
    parts = rng.standard_normal((splits, mats, M, N)).astype(np.float32)
    missing = np.repeat(rng.random((M, N // 4)) < 0.2, 4, axis=1)
    missing[0, :4], missing[0, 4:8] = True, False
    for m, n in np.argwhere(missing[:, ::4]):
        parts[rng.integers(splits), 0, m, 4 * n] = np.nan
    total = np.zeros((mats, M, N), np.float32)
    for p in parts:
        total = total + p
    Y = outputs((M, N), 1 if mats == 1 else 3)
    p = on_device(parts, kernels.no_part())
    assert kernels.dense_finish(p.data_ptr(), *[t.data_ptr() for t in Y], *[None] * (3 - len(Y)), M, N, splits,
                                kind) == 0
    check(Y, total, missing)
