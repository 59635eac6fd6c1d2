"""Host-side checks of the products over quantized weights (no GPU): what the C calls refuse, before any
CUDA call (the fake pointers are never dereferenced), the sizes they ask for, and what the binding
refuses."""
import ctypes
import subprocess
import sys

import pytest
import torch

import calibration_free_weight_hqq_b200 as hqq

OK, INVALID, UNSUPPORTED, SHAPE, ALIGN, CUDA, WORKSPACE = range(7)
FAKE, ODD = 0x100000, 0x100008  # 16-byte aligned and not
BF16, F16, F32 = hqq.HQQ_BF16, hqq.HQQ_F16, hqq.HQQ_F32


@pytest.fixture(scope="module")
def L():
    return hqq.lib()


def weight(rows=256, cols=512, nbits=4, G=64, axis=1, meta=torch.bfloat16, quant=False, flags=0, **kw):
    p = hqq.make_params(nbits, G, axis, w_dtype=torch.bfloat16, meta_dtype=meta, quant_scale=quant,
                        quant_zero=quant, meta_group_size=kw.pop("run", 128))
    p.flags = flags
    f = dict(Wq_packed=FAKE, scale=FAKE, zero=FAKE, scale_mm=FAKE if quant else None,
             zero_mm=FAKE if quant else None, bias=None)
    f.update(kw)
    return hqq.HQQWeight(*(f[n] for n, _ in hqq.HQQWeight._fields_[:6]), rows, cols, p)


def linear(L, w, X=FAKE, M=4, dt=BF16, Y=FAKE, ws=FAKE, n=1 << 40):
    return L.hqq_linear_ex(X, M, dt, ctypes.addressof(w), Y, ws, n, None)


def grad(L, w, dY=FAKE, M=4, dt=BF16, dX=FAKE, db=None, ws=FAKE, n=1 << 40):
    return L.hqq_linear_backward(dY, M, dt, ctypes.addressof(w), dX, db, ws, n, None)


def gated(L, g, u, X=FAKE, M=4, dt=BF16, act=0, Y=FAKE, G=None, U=None, ws=FAKE, n=1 << 40):
    return L.hqq_gated_linear(X, M, dt, ctypes.addressof(g), ctypes.addressof(u), act, Y, G, U, ws, n,
                              None)


def gated_grad(L, g, u, dY=FAKE, G=FAKE, U=FAKE, M=4, dt=BF16, act=0, dG=FAKE, dU=FAKE, dX=FAKE,
               dbg=None, dbu=None, ws=FAKE, n=1 << 40):
    return L.hqq_gated_linear_backward(dY, G, U, M, dt, ctypes.addressof(g), ctypes.addressof(u), act,
                                       dG, dU, dX, dbg, dbu, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nbits=5), UNSUPPORTED), (dict(G=48), UNSUPPORTED), (dict(axis=2), UNSUPPORTED),
    (dict(rows=-8), INVALID), (dict(cols=500), SHAPE), (dict(rows=252), SHAPE),
    (dict(rows=100, axis=0, G=64), SHAPE), (dict(cols=516, axis=0), SHAPE),
    (dict(rows=1 << 31, cols=64), SHAPE), (dict(flags=4), INVALID),
    (dict(quant=True, run=4), UNSUPPORTED), (dict(quant=True, scale_mm=None), INVALID),
    (dict(quant=True, zero_mm=None), INVALID), (dict(Wq_packed=None), INVALID),
    (dict(scale=None), INVALID), (dict(zero=None), INVALID), (dict(Wq_packed=ODD), ALIGN),
    (dict(scale=FAKE + 1), ALIGN), (dict(zero=FAKE + 2, meta=torch.float32), ALIGN),
    (dict(quant=True, zero_mm=FAKE + 4), ALIGN), (dict(bias=FAKE + 1), ALIGN),
])
def test_bad_weights_are_refused_by_every_call(L, kw, status):
    bad, good = weight(**kw), weight()
    assert linear(L, bad) == grad(L, bad) == status
    assert gated(L, bad, good) == gated(L, good, bad) == status
    assert gated_grad(L, bad, good) == gated_grad(L, good, bad) == status
    assert L.hqq_linear_workspace_bytes(4, ctypes.addressof(bad), 0) == ctypes.c_size_t(-1).value
    assert L.hqq_gated_linear_workspace_bytes(4, ctypes.addressof(good), ctypes.addressof(bad), 1) == \
        ctypes.c_size_t(-1).value


def test_null_weights_and_bad_meta_dtype(L):
    w = weight()
    assert L.hqq_linear_ex(FAKE, 4, BF16, None, FAKE, FAKE, 1 << 40, None) == INVALID
    assert L.hqq_linear_backward(FAKE, 4, BF16, None, FAKE, None, FAKE, 1 << 40, None) == INVALID
    assert L.hqq_gated_linear(FAKE, 4, BF16, ctypes.addressof(w), None, 0, FAKE, None, None, FAKE,
                              1 << 40, None) == INVALID
    w.params.meta_dtype = 7
    assert linear(L, w) == UNSUPPORTED


@pytest.mark.parametrize("call", ["linear", "grad", "gated", "gated_grad"])
def test_bad_calls(L, call):
    w = weight()
    f = {"linear": lambda **k: linear(L, w, **k), "grad": lambda **k: grad(L, w, **k),
         "gated": lambda **k: gated(L, w, w, **k), "gated_grad": lambda **k: gated_grad(L, w, w, **k)}[call]
    back = call.endswith("grad")
    x, y = ("dY", "dX") if back else ("X", "Y")
    assert f(M=-1) == INVALID and f(M=1 << 31) == SHAPE
    assert f(dt=F32) == f(dt=9) == UNSUPPORTED
    assert f(**{x: None}) == f(**{y: None}) == INVALID
    assert f(**{x: ODD}) == f(**{y: ODD}) == ALIGN
    M = 1 << 12  # enough tokens to need a workspace
    need = (L.hqq_gated_linear_workspace_bytes(M, ctypes.addressof(w), ctypes.addressof(w), int(back))
            if "gated" in call else L.hqq_linear_workspace_bytes(M, ctypes.addressof(w), int(back)))
    assert 0 < need < 1 << 40
    assert f(M=M, ws=None) == f(M=M, n=need - 1) == WORKSPACE
    assert f(M=M, ws=ODD) == ALIGN
    if "gated" in call:
        assert f(act=3) == f(act=-1) == UNSUPPORTED
        outs = ("dG", "dU", "G", "U") if back else ("G", "U")
        for o in outs:
            assert f(**{o: ODD}) == ALIGN
        if back:
            assert f(dG=None) == f(U=None) == INVALID
            assert f(dbg=FAKE + 1) == ALIGN
        other = weight(rows=264)
        assert (gated_grad(L, w, other) if back else gated(L, w, other)) == SHAPE
    elif back:
        assert f(db=FAKE + 1) == ALIGN


def test_nothing_to_do_needs_no_pointers(L):
    w = weight(Wq_packed=FAKE)
    assert linear(L, w, M=0, X=None, Y=None, ws=None, n=0) == OK
    assert grad(L, w, M=0, dY=None, dX=None, ws=None, n=0) == OK
    assert gated(L, w, w, M=0, X=None, Y=None, ws=None, n=0) == OK
    assert gated_grad(L, w, w, M=0, dY=None, G=None, U=None, dG=None, dU=None, dX=None, ws=None, n=0) == OK
    none = weight(rows=0, Wq_packed=None, scale=None, zero=None)
    assert linear(L, none, Y=None, ws=None, n=0) == OK
    empty = weight(cols=0, Wq_packed=None, scale=None, zero=None)
    assert grad(L, empty, dX=None, ws=None, n=0) == OK


def test_workspace_sizes(L):
    def one(M, back, **kw):
        return L.hqq_linear_workspace_bytes(M, ctypes.addressof(weight(**kw)), back)

    assert one(0, 0) == one(0, 1) == 0
    for M in range(1, 9):
        assert one(M, 0) == 0                       # a few tokens: straight from the codes
        assert one(M, 0, nbits=3, cols=72, G=8) == 0
    big = dict(rows=4096, cols=4096)
    assert one(8192, 0, **big) == one(8192, 1, **big) == 2 * 4096 * 4096  # the dequantized weight
    # few tiles: also the partial sums of four parts of the contraction
    assert one(1, 0, axis=0, **big) == 2 * 4096 * 4096 + 4 * 4 * 4096
    a, b = weight(**big), weight(nbits=2, G=16, **big)
    size = L.hqq_gated_linear_workspace_bytes
    assert size(1, ctypes.addressof(a), ctypes.addressof(a), 0) == 0
    # two formats: both dequantized, and two parts of both products
    assert size(1, ctypes.addressof(a), ctypes.addressof(b), 0) == 4 * 4096 * 4096 + 2 * 2 * 4 * 4096
    assert size(8192, ctypes.addressof(a), ctypes.addressof(a), 1) == 4 * 4096 * 4096
    assert 0 < one(64, 0, **big) < 2 * 4096 * 4096   # partial sums only
    assert one(-1, 0) == one(1 << 31, 0) == ctypes.c_size_t(-1).value


def test_binding_refuses_host_tensors_and_wrong_shapes():
    with pytest.raises(ValueError):
        hqq.quantized_weight((torch.zeros(4, dtype=torch.uint8), torch.zeros(1), torch.zeros(1)), 8, 64,
                             hqq.make_params(1, 64, 1))
    with pytest.raises(hqq.HQQError):
        hqq.quantized_weight((None, None, None), 8, 60, hqq.make_params(4, 64, 1))
    w = hqq.QuantizedWeight(8, 64, torch.device("cuda", 0), None, [], weight(rows=8, cols=64))
    for call in (lambda t: hqq.hqq_linear_ex(t, w), lambda t: hqq.hqq_linear_backward(t, w),
                 lambda t: hqq.hqq_gated_linear(t, w, w),
                 lambda t: hqq.hqq_gated_linear_backward(t, t, t, w, w)):
        with pytest.raises(ValueError):
            call(torch.zeros(1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        hqq.hqq_gated_linear(torch.zeros(1, 64), w, w, "relu")


def test_struct_mirror_matches_the_header():
    """The struct's size: six pointers, two 64-bit sizes and hqq_params (13 4-byte fields), padded."""
    assert ctypes.sizeof(hqq.HQQParams) == 52
    assert ctypes.sizeof(hqq.HQQWeight) == 6 * 8 + 2 * 8 + 56


def test_overlapping_tensors_are_refused(L):
    """An output may overlap neither activations, nor the workspace, nor another output."""
    w = weight(rows=256, cols=512, axis=0)       # dequantized: it needs a workspace
    M, MB = 4, 1 << 20
    far = [FAKE + i * 64 * MB for i in range(12)]
    for back in range(-4 * 256 * 2 + 16, 4 * 512 * 2, 512):      # X [4, 512] against Y [4, 256]
        assert linear(L, w, X=far[0], Y=far[0] + back, ws=far[1]) == INVALID
    assert linear(L, w, X=far[0], Y=far[1], ws=far[1] + 1024) == INVALID
    assert grad(L, w, dY=far[0], dX=far[0], ws=far[1]) == INVALID
    assert grad(L, w, dY=far[0], dX=far[2], db=far[2] + 16, ws=far[1]) == INVALID
    assert gated(L, w, w, X=far[0], Y=far[1], G=far[1], U=far[2], ws=far[3]) == INVALID
    assert gated(L, w, w, X=far[0], Y=far[1], G=far[2], U=far[0], ws=far[3]) == INVALID
    names = ("dY", "G", "U", "dG", "dU", "dX", "dbg", "dbu", "ws")
    apart = dict(zip(names, far))
    for out in ("dG", "dU", "dX", "dbg", "dbu", "ws"):
        for other in names:
            if other != out:
                assert gated_grad(L, w, w, **{**apart, out: apart[other]}) == INVALID, (out, other)
    # apart, and touching end to start: only the device is missing
    end = FAKE + M * 512 * 2
    assert linear(L, w, X=FAKE, Y=end, ws=far[1]) == linear(L, w, X=far[0], Y=far[2], ws=far[1]) != INVALID
    assert gated_grad(L, w, w, **apart) != INVALID
    # the same token tensor as two inputs, and one weight as gate and up, are fine
    assert gated_grad(L, w, w, **{**apart, "G": apart["dY"], "U": apart["dY"]}) != INVALID


def test_the_package_imports_with_a_torch_that_has_no_cuda():
    """Such a torch lacks the CUDA functions of torch._C; a call then refuses its tensors."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_getCurrent")]:
    delattr(torch._C, name)
import calibration_free_weight_hqq_b200 as hqq
t = torch.zeros(1, 64, dtype=torch.bfloat16)
try:
    hqq.quantized_weight((t, t, t), 8, 64, hqq.make_params(1, 64, 1))
except ValueError as e:
    print("refused:", e)
"""
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "refused:" in run.stdout, run.stderr
