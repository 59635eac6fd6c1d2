"""The products over quantized weights (hqq_linear_ex, hqq_linear_backward, hqq_gated_linear,
hqq_gated_linear_backward) against the oracle's W' and 64-bit products.

Inputs: codes, scale and zero are drawn here and packed by the oracle; activations come from a
seeded generator. W' is the oracle's dequantized weight rounded once to the activation type.

Bars (u: half a step of the output type, 2^-8 bf16, 2^-11 fp16; fp16 also 2^-25 absolute where
its results are subnormal):
  * one-hot rows select single weights: each output is one product with 1, exact in any
    accumulation, so outputs must equal W' bit for bit (forward and backward).
  * a sum of L products: u |S| + (1 + u) e, e = L 2^-23 sum|terms| (fp32 accumulation in any
    order, truncation allowed inside the tensor core), plus 2^-23 (|S| + |bias|) of the bias add.
  * act: the special-function exponential is off by 2 + 1.173 |x| ulp (its documented bound), the
    quotient by 2 ulp: under 32 ulp = 2^-18 for |x| <= 20. gelu: erfc is off by 4 ulp, its
    argument's rounding is amplified by 2 x^2 <= 64 for |g| <= 8: under 2^-17. tanh form: the
    argument 2y (|2y| <= 70 for |g| <= 8, 6 roundings) enters an exponential: (6 * 70 / 2 + 90)
    2^-23 < 2^-14. Below |g| = 8 in the lower tail act is under 1e-13: an absolute 1e-12.
  * act': a sum of terms of at most 8 in size under the same errors: 2^-13 |g|-free absolute bound
    for the tanh form, 2^-15 for the others.
"""
import threading
import warnings

import numpy as np
import pytest
import torch

import calibration_free_weight_hqq_b200 as hqq
import oracle

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-37, "f16": 2.0 ** -25}
ACT_REL = {"silu": 2.0 ** -18, "gelu": 2.0 ** -17, "gelu_tanh": 2.0 ** -14}
GRAD_ABS = {"silu": 2.0 ** -15, "gelu": 2.0 ** -15, "gelu_tanh": 2.0 ** -13}

NBITS = (8, 4, 3, 2, 1)


class Layer:
    """A drawn weight [N, K]: its handle, and W' (float64 array of dtype's values)."""

    def __init__(self, N, K, nbits=4, G=64, axis=1, dtype="bf16", meta="bf16", bias=False, seed=0,
                 run=128):
        rng = np.random.default_rng(seed)
        ng = N * K // G
        codes = rng.integers(0, 2 ** nbits, size=N * K, dtype=np.uint8)
        scale = (rng.random(ng) * 0.02 + 1e-3).astype(np.float32)
        zero = (rng.random(ng) * (2 ** nbits - 1)).astype(np.float32)
        q = {"Wq_packed": torch.from_numpy(oracle.pack(codes, nbits)).cuda()}
        quant = {"u8": (True, True), "u8scale": (True, False), "u8zero": (False, True)}
        qs, qz = quant.get(meta, (False, False))
        plain = "f32" if meta == "f32" else "f16" if meta == "f16" else "bf16"
        vals = {}
        for name, v, is8 in (("scale", scale, qs), ("zero", zero, qz)):
            if is8:
                c, mm = oracle.quantize_meta(v, run)
                vals[name] = oracle.dequantize_meta(c, mm, run)
                q[name], q[name + "_mm"] = torch.from_numpy(c).cuda(), torch.from_numpy(mm).cuda()
            else:
                vals[name] = oracle.round_to_dtype(v, plain)
                q[name] = torch.from_numpy(vals[name]).to(TORCH[plain]).cuda()
        self.N, self.K, self.dtype = N, K, dtype
        W = oracle.dequantize(codes, vals["scale"], vals["zero"], N, K, G, axis)
        self.W = oracle.round_to_dtype(W, dtype).astype(np.float64)
        self.bias = None
        b = None
        if bias:
            self.bias = oracle.round_to_dtype(rng.standard_normal(N).astype(np.float32), dtype)
            b = torch.from_numpy(self.bias).to(TORCH[dtype]).cuda()
            self.bias = self.bias.astype(np.float64)
        self.params = hqq.make_params(nbits, G, axis, w_dtype=TORCH[dtype],
                                      meta_dtype=TORCH[plain], quant_scale=qs, quant_zero=qz,
                                      meta_group_size=run)
        self.h = hqq.quantized_weight(q, N, K, self.params, bias=b)

    def project(self, X):
        """(X W'^T + bias, its fp32 error bound) in 64 bits."""
        S = X @ self.W.T
        e = max(self.K, 1) * 2.0 ** -23 * (np.abs(X) @ np.abs(self.W).T)
        if self.bias is not None:
            S = S + self.bias
            e = e + 2.0 ** -23 * (np.abs(S) + np.abs(self.bias))
        return S, e


def draw(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(shape, generator=g) * scale).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def close(got, want, err, dtype, what):
    u = UNIT[dtype]
    tol = u * np.abs(want) + (1 + u) * err + TINY[dtype]
    assert np.isfinite(got).all(), what
    worst = (np.abs(got - want) / tol).max() if want.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def act64(name, g):
    import math
    if name == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        erfc = np.vectorize(math.erfc)
        c = 0.5 * erfc(-g / math.sqrt(2))
        return g * c, c + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * k * (1 + 3 * 0.044715 * g * g)


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert hqq.hqq_wait_timeouts() == 0


# ------------------------------------------------------------------ W' bit for bit

FORMATS = [(b, G, axis, meta) for b in NBITS
           for G, axis, meta in ((8, 1, "bf16"), (16, 1, "bf16"), (32, 1, "f32"), (64, 1, "bf16"),
                                 (128, 1, "f16"), (64, 1, "u8"), (16, 1, "u8"), (64, 1, "u8scale"),
                                 (256, 1, "u8zero"), (8, 0, "bf16"), (64, 0, "u8"))]


@pytest.mark.parametrize("nbits,G,axis,meta", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_hot_forward_is_the_dequantized_weight(nbits, G, axis, meta, dtype):
    N = 72 if axis == 1 else 2 * max(G, 32)
    K = 3 * G if G >= 64 else 11 * G if axis == 1 else 136
    L = Layer(N, K, nbits, G, axis, dtype, meta, seed=nbits * 100 + G)
    eye = torch.eye(K, dtype=TORCH[dtype], device="cuda")
    whole = host(hqq.hqq_linear_ex(eye, L.h))           # many tokens
    assert np.array_equal(whole, L.W.T)
    for k0 in range(0, K, 24):                          # few tokens
        assert np.array_equal(host(hqq.hqq_linear_ex(eye[k0:k0 + 24], L.h)), L.W.T[k0:k0 + 24])
    for k0 in range(0, K, 7):
        assert np.array_equal(host(hqq.hqq_linear_ex(eye[k0:k0 + 7], L.h)), L.W.T[k0:k0 + 7])


@pytest.mark.parametrize("nbits,G,axis,meta", FORMATS)
def test_one_hot_backward_is_the_dequantized_weight(nbits, G, axis, meta):
    N = 328 if axis == 1 else 5 * max(G, 64)
    K = 2 * G if G >= 64 else 9 * G if axis == 1 else 136
    L = Layer(N, K, nbits, G, axis, "bf16", meta, seed=nbits * 100 + G + 1)
    eye = torch.eye(N, dtype=torch.bfloat16, device="cuda")
    assert np.array_equal(host(hqq.hqq_linear_backward(eye, L.h)), L.W)


@pytest.mark.parametrize("K", [8, 136, 264])
@pytest.mark.parametrize("G,meta,dtype", [(16, "f16", "bf16"), (32, "u8", "f16"), (64, "f32", "f16"),
                                          (128, "u8scale", "bf16"), (256, "u8zero", "f16")])
@pytest.mark.parametrize("nbits", NBITS)
def test_one_hot_of_groups_down_the_columns(nbits, G, meta, dtype, K):
    N = 3 * G
    L = Layer(N, K, nbits, G, 0, dtype, meta, seed=nbits + G + K)
    eye = torch.eye(K, dtype=TORCH[dtype], device="cuda")
    assert np.array_equal(host(hqq.hqq_linear_ex(eye, L.h)), L.W.T)
    eye = torch.eye(N, dtype=TORCH[dtype], device="cuda")
    assert np.array_equal(host(hqq.hqq_linear_backward(eye, L.h)), L.W)


# ------------------------------------------------------------------ random products

SIZES = [(1, 8, 8), (1, 4096, 1024), (2, 264, 320), (7, 40, 72), (8, 1000, 2048), (9, 136, 1096),
         (16, 512, 4096), (17, 72, 640), (31, 24, 128), (32, 264, 256), (33, 264, 256),
         (100, 520, 192), (128, 256, 64), (129, 8, 4104), (257, 776, 328), (600, 1032, 520)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("nbits,dtype,meta", [(4, "bf16", "bf16"), (2, "f16", "f32"),
                                              (3, "bf16", "u8"), (8, "f16", "f16")])
def test_linear_ex(M, N, K, nbits, dtype, meta):
    G = 64 if K % 64 == 0 else 8
    L = Layer(N, K, nbits, G, 1, dtype, meta, bias=nbits != 4, seed=M + N + K)
    X, X64 = draw((M, K), M, dtype)
    S, e = L.project(X64)
    close(host(hqq.hqq_linear_ex(X, L.h)), S, e, dtype, "Y")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("nbits,dtype,axis", [(4, "bf16", 1), (1, "f16", 1), (3, "bf16", 0)])
def test_linear_backward(M, N, K, nbits, dtype, axis):
    if axis == 1:
        G = 64 if K % 64 == 0 else 8
    else:
        G = 64 if N % 64 == 0 else 8
    L = Layer(N, K, nbits, G, axis, dtype, seed=M + N + K)
    dY, dY64 = draw((M, N), M + 1, dtype)
    dX, db = hqq.hqq_linear_backward(dY, L.h, bias_grad=True)
    e = N * 2.0 ** -23 * (np.abs(dY64) @ np.abs(L.W))
    close(host(dX), dY64 @ L.W, e, dtype, "dX")
    close(host(db), dY64.sum(0), M * 2.0 ** -23 * np.abs(dY64).sum(0), dtype, "dbias")


def check_gated(M, N, K, act, dtype, gate, up, X, X64):
    Y, G, U = hqq.hqq_gated_linear(X, gate.h, up.h, act, save=True)
    g, eg = gate.project(X64)
    u, eu = up.project(X64)
    assert np.abs(g).max() < (20 if act == "silu" else 8)
    a, _ = act64(act, g)
    close(host(G), g, eg, dtype, "G")
    close(host(U), u, eu, dtype, "U")
    ea = 1.2 * eg + ACT_REL[act] * np.abs(a) + 1e-12  # |act'| < 1.2
    close(host(Y), a * u, ea * np.abs(u) + (np.abs(a) + ea) * eu + 2.0 ** -23 * np.abs(a * u), dtype,
          "Y")
    again = hqq.hqq_gated_linear(X, gate.h, up.h, act)
    assert torch.equal(again, Y)  # the same with and without G and U
    return Y, G, U


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("nbits,dtype,act,bias", [(4, "bf16", "silu", False),
                                                  (2, "f16", "gelu", True),
                                                  (3, "bf16", "gelu_tanh", True)])
def test_gated(M, N, K, nbits, dtype, act, bias):
    G = 64 if K % 64 == 0 else 8
    gate = Layer(N, K, nbits, G, 1, dtype, bias=bias, seed=M + N + K)
    up = Layer(N, K, nbits, G, 1, dtype, bias=bias, seed=M + N + K + 1)
    # scaled so that |g| stays under 8
    X, X64 = draw((M, K), M, dtype, scale=0.5 / np.sqrt(K) / np.abs(gate.W).max())
    check_gated(M, N, K, act, dtype, gate, up, X, X64)


@pytest.mark.parametrize("M", [1, 20, 70])
def test_gated_of_two_formats(M):
    N, K = 128, 256
    gate = Layer(N, K, 4, 64, 1, "bf16", "bf16", seed=1)
    for kw in (dict(nbits=2, G=16), dict(nbits=4, G=32), dict(nbits=4, G=64, axis=0),
               dict(nbits=4, G=64, meta="f32"), dict(nbits=4, G=64, meta="u8")):
        up = Layer(N, K, dtype="bf16", seed=2, **kw)
        X, X64 = draw((M, K), M, "bf16", scale=0.1)
        check_gated(M, N, K, "silu", "bf16", gate, up, X, X64)


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 264, 136), (130, 520, 328), (300, 776, 512)])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("f16", "gelu"), ("bf16", "gelu_tanh")])
def test_gated_backward(M, N, K, dtype, act):
    G = 64 if K % 64 == 0 else 8
    gate = Layer(N, K, 4, G, 1, dtype, seed=M + N)
    up = Layer(N, K, 2, 8, 1, dtype, meta="u8", seed=M + N + 1)
    dY, dY64 = draw((M, N), 1, dtype)
    g, g64 = draw((M, N), 2, dtype, 1.5)
    u, u64 = draw((M, N), 3, dtype)
    dX, dG, dU, dbg, dbu = hqq.hqq_gated_linear_backward(dY, g, u, gate.h, up.h, act,
                                                         bias_grad=True)
    a, d = act64(act, g64)
    close(host(dG), dY64 * u64 * d, np.abs(dY64 * u64) * GRAD_ABS[act], dtype, "dG")
    close(host(dU), dY64 * a, np.abs(dY64) * (2 * ACT_REL[act] * np.abs(a) + 1e-12), dtype, "dU")
    rG, rU = host(dG), host(dU)
    S = np.abs(rG) @ np.abs(gate.W) + np.abs(rU) @ np.abs(up.W)
    close(host(dX), rG @ gate.W + rU @ up.W, 2 * N * 2.0 ** -23 * S, dtype, "dX")
    close(host(dbg), rG.sum(0), M * 2.0 ** -23 * np.abs(rG).sum(0), dtype, "dbias_gate")
    close(host(dbu), rU.sum(0), M * 2.0 ** -23 * np.abs(rU).sum(0), dtype, "dbias_up")


# ------------------------------------------------------------------ dequantized weights (axis 0)

@pytest.mark.parametrize("M,N,K", [(9, 64, 72), (33, 264, 256), (128, 256, 64), (257, 776, 328),
                                   (600, 1032, 520), (2500, 264, 136)])
@pytest.mark.parametrize("dtype,act,bias", [("bf16", "silu", True), ("f16", "gelu", False),
                                            ("bf16", "gelu_tanh", False)])
def test_groups_down_the_columns(M, N, K, dtype, act, bias):
    gate = Layer(N, K, 4, 8, 0, dtype, bias=bias, seed=M + N)
    up = Layer(N, K, 4, 8, 0, dtype, bias=bias, seed=M + N + 1)
    X, X64 = draw((M, K), M, dtype, scale=0.5 / np.sqrt(K) / np.abs(gate.W).max())
    S, e = up.project(X64)
    close(host(hqq.hqq_linear_ex(X, up.h)), S, e, dtype, "Y")
    check_gated(M, N, K, act, dtype, gate, up, X, X64)


@pytest.mark.parametrize("M,N,K", [(2304, 2048, 2048), (4100, 1032, 4096)])
def test_many_tokens_along_the_rows(M, N, K):
    """Enough work that the weight is dequantized once; checked on sampled tokens."""
    gate, up = (Layer(N, K, 4, 64, 1, "bf16", seed=s) for s in (1, 2))
    X, X64 = draw((M, K), 3, "bf16", scale=0.02)
    rows = np.r_[0:3, M // 2:M // 2 + 3, M - 3:M]
    Y, G, U = hqq.hqq_gated_linear(X, gate.h, up.h, save=True)
    g, eg = gate.project(X64[rows])
    u, eu = up.project(X64[rows])
    a, _ = act64("silu", g)
    assert np.abs(g).max() < 20
    close(host(G)[rows], g, eg, "bf16", "G")
    close(host(U)[rows], u, eu, "bf16", "U")
    ea = 1.2 * eg + ACT_REL["silu"] * np.abs(a) + 1e-12
    close(host(Y)[rows], a * u, ea * np.abs(u) + (np.abs(a) + ea) * eu + 2.0 ** -23 * np.abs(a * u),
          "bf16", "Y")
    S, e = up.project(X64[rows])
    close(host(hqq.hqq_linear_ex(X, up.h))[rows], S, e, "bf16", "Y of one weight")
    dY, dY64 = draw((M, N), 4, "bf16")
    dX = host(hqq.hqq_linear_backward(dY, gate.h))[rows]
    close(dX, dY64[rows] @ gate.W, N * 2.0 ** -23 * (np.abs(dY64[rows]) @ np.abs(gate.W)), "bf16", "dX")


@pytest.mark.parametrize("M,N,K", [(5, 264, 4104), (129, 520, 2304), (300, 72, 8192)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_few_tiles_of_a_long_contraction(M, N, K, act):
    """Products on dequantized weights whose contraction is cut into parts."""
    gate = Layer(N, K, 4, 8, 0, "bf16", bias=True, seed=M)
    up = Layer(N, K, 2, 8, 0, "bf16", seed=M + 1)
    X, X64 = draw((M, K), M, "bf16", scale=0.5 / np.sqrt(K) / np.abs(gate.W).max())
    check_gated(M, N, K, act, "bf16", gate, up, X, X64)
    S, e = gate.project(X64)
    close(host(hqq.hqq_linear_ex(X, gate.h)), S, e, "bf16", "Y")
    gate, up = (Layer(K, N, 4, 8, 0, "bf16", seed=M + s) for s in (2, 3))  # gradients contract over K
    dY, _ = draw((M, K), 1, "bf16")
    g, _ = draw((M, K), 2, "bf16")
    u, _ = draw((M, K), 3, "bf16")
    dX, dG, dU = hqq.hqq_gated_linear_backward(dY, g, u, gate.h, up.h, act)
    rG, rU = host(dG), host(dU)
    S = np.abs(rG) @ np.abs(gate.W) + np.abs(rU) @ np.abs(up.W)
    close(host(dX), rG @ gate.W + rU @ up.W, 2 * K * 2.0 ** -23 * S, "bf16", "dX")
    e = K * 2.0 ** -23 * (np.abs(host(dY)) @ np.abs(gate.W))
    close(host(hqq.hqq_linear_backward(dY, gate.h)), host(dY) @ gate.W, e, "bf16", "dX of one weight")


# ------------------------------------------------------------------ odd scales and zeros

@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("meta", ["same", "f32"])
def test_one_hot_with_odd_scales_and_zeros(nbits, dtype, meta):
    """Zeros next to 0, negative, far outside the codes and far beyond them; scale 0 and tiny."""
    N, K, G = 32, 320, 64
    rng = np.random.default_rng(nbits)
    codes = rng.integers(0, 2 ** nbits, size=N * K, dtype=np.uint8)
    ng = N * K // G
    zero = rng.choice([0.0, -0.0, 1e-3, -1e-3, 0.37, 7.5, -5.0, 123.0, -1000.0, 4097.0, 3e4, 1e-7], ng)
    scale = rng.choice([0.0, 1e-4, 0.01, 1.0, -0.5, 3e-6], ng)
    kind = dtype if meta == "same" else "f32"
    zero = oracle.round_to_dtype(zero.astype(np.float32), kind)
    scale = oracle.round_to_dtype(scale.astype(np.float32), kind)
    W = oracle.round_to_dtype(oracle.dequantize(codes, scale, zero, N, K, G, 1), dtype)
    prm = hqq.make_params(nbits, G, 1, w_dtype=TORCH[dtype], meta_dtype=TORCH[kind])
    q = [torch.from_numpy(oracle.pack(codes, nbits)).cuda()] + \
        [torch.from_numpy(v).to(TORCH[kind]).cuda() for v in (scale, zero)]
    w = hqq.quantized_weight(q, N, K, prm)
    eye = torch.eye(K, dtype=TORCH[dtype], device="cuda")
    for n in (8, 40):
        for k0 in range(0, K, n):
            got = host(hqq.hqq_linear_ex(eye[k0:k0 + n], w))
            assert np.array_equal(got, W.T[k0:k0 + n].astype(np.float64))
    got = host(hqq.hqq_linear_backward(torch.eye(N, dtype=TORCH[dtype], device="cuda"), w))
    assert np.array_equal(got, W.astype(np.float64))


@pytest.mark.parametrize("run", [8, 24, 100, 1024])
def test_second_level_runs(run):
    for M in (3, 50):
        L = Layer(136, 448, 4, 64, 1, "bf16", "u8", seed=run, run=run)
        X, X64 = draw((M, 448), run, "bf16")
        S, e = L.project(X64)
        close(host(hqq.hqq_linear_ex(X, L.h)), S, e, "bf16", "Y")
        dY, dY64 = draw((M, 136), run, "bf16")
        e = 136 * 2.0 ** -23 * (np.abs(dY64) @ np.abs(L.W))
        close(host(hqq.hqq_linear_backward(dY, L.h)), dY64 @ L.W, e, "bf16", "dX")


def test_meta_and_bias_views_of_natural_alignment():
    """Scale, zero and bias that start on an odd element."""
    N, K = 72, 320
    L = Layer(N, K, 4, 64, 1, "bf16", bias=True, seed=9)

    def shifted(t):
        big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        big[1:] = t.reshape(-1)
        return big[1:]

    pk, sc, zr = L.h.tensors[:3]
    w = hqq.quantized_weight((pk, shifted(sc), shifted(zr)), N, K, L.params,
                             bias=shifted(L.h.tensors[-1]))
    for M in (1, 40):
        X, _ = draw((M, K), M, "bf16")
        assert torch.equal(hqq.hqq_linear_ex(X, w), hqq.hqq_linear_ex(X, L.h))


# ------------------------------------------------------------------ infinities, empty, untouched rows

@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("axis", [1, 0])
def test_a_token_of_infinities_stays_alone(M, axis):
    L = Layer(264, 320, 4, 8, axis, "bf16", seed=2)
    X, _ = draw((M, 320), 1, "bf16")
    clean = hqq.hqq_linear_ex(X, L.h)
    X[2, 7], X[3, 0] = float("inf"), float("nan")
    got = hqq.hqq_linear_ex(X, L.h)
    keep = [m for m in range(M) if m not in (2, 3)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[2]).any()
    dY, _ = draw((M, 264), 1, "bf16")
    clean = hqq.hqq_linear_backward(dY, L.h)
    dY[2, 7] = float("inf")
    got = hqq.hqq_linear_backward(dY, L.h)
    keep = [m for m in range(M) if m != 2]
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[2]).any()


@pytest.mark.parametrize("M", [3, 40])
def test_a_feature_of_infinite_scale_stays_alone(M):
    N, K = 40, 256
    L = Layer(N, K, 4, 64, 1, "bf16", seed=2)
    X, _ = draw((M, K), 1, "bf16")
    clean = hqq.hqq_linear_ex(X, L.h)
    L.h.tensors[1].view(N, -1)[5, 1] = float("inf")
    got = hqq.hqq_linear_ex(X, L.h)
    keep = [n for n in range(N) if n != 5]
    assert torch.equal(got[:, keep], clean[:, keep]) and not torch.isfinite(got[:, 5]).any()


@pytest.mark.parametrize("M", [0, 1, 8, 9, 100, 300])
def test_rows_behind_the_last_token_stay_as_they_were(M):
    N, K = 136, 192
    gate, up = (Layer(N, K, 4, 64, 1, "bf16", seed=s) for s in (1, 2))
    X, _ = draw((max(M, 1), K), 1, "bf16")
    X = X[:M]
    bufs = [torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    Y, G, U, dG, dU = (b[:M] for b in bufs)
    last = torch.full((M + 3, K), 7.0, dtype=torch.bfloat16, device="cuda")
    hqq.hqq_gated_linear(X, gate.h, up.h, Y=Y, G=G, U=U)
    hqq.hqq_gated_linear_backward(Y, G, U, gate.h, up.h, dX=last[:M], dG=dG, dU=dU)
    torch.cuda.synchronize()
    for b in (*bufs, last):
        assert (b[M:] == 7.0).all()
        assert not (b[:M] == 7.0).all() or M == 0


@pytest.mark.parametrize("axis", [1, 0])
def test_empty_shapes(axis):
    bf = dict(dtype=torch.bfloat16, device="cuda")
    L = Layer(64, 64, 4, 64, axis, "bf16", bias=True, seed=1)
    assert hqq.hqq_linear_ex(torch.empty(0, 64, **bf), L.h).shape == (0, 64)
    dX, db = hqq.hqq_linear_backward(torch.empty(0, 64, **bf), L.h, bias_grad=True)
    assert dX.shape == (0, 64) and (db == 0).all()
    out = hqq.hqq_gated_linear_backward(*[torch.empty(0, 64, **bf)] * 3, L.h, L.h, bias_grad=True)
    assert [tuple(t.shape) for t in out] == [(0, 64)] * 3 + [(64,)] * 2
    assert (out[3] == 0).all() and (out[4] == 0).all()
    # no input features: every sum is the bias
    none = torch.empty(0, **bf)
    prm = hqq.make_params(4, 64, axis, w_dtype=torch.bfloat16)
    b = torch.randn(64, device="cuda").bfloat16()
    w = hqq.quantized_weight((torch.empty(0, dtype=torch.uint8, device="cuda"), none, none), 64, 0,
                             prm, bias=b)
    for M in (1, 70000):
        X = torch.empty(M, 0, **bf)
        assert torch.equal(hqq.hqq_linear_ex(X, w), b.expand(M, 64))
        Y, G, U = hqq.hqq_gated_linear(X, w, w, save=True)
        assert torch.equal(G, b.expand(M, 64)) and torch.equal(U, G)
    dY = torch.randn(5, 64, device="cuda").bfloat16()
    dX, db = hqq.hqq_linear_backward(dY, w, bias_grad=True)
    assert dX.shape == (5, 0)
    close(host(db), host(dY).sum(0), 5 * 2.0 ** -23 * np.abs(host(dY)).sum(0), "bf16", "dbias")
    # no output features: nothing forward, an empty sum back
    w = hqq.quantized_weight((torch.empty(0, dtype=torch.uint8, device="cuda"), none, none), 0, 64, prm)
    assert hqq.hqq_linear_ex(torch.empty(3, 64, **bf), w).shape == (3, 0)
    assert (hqq.hqq_linear_backward(torch.empty(3, 0, **bf), w) == 0).all()
    assert (hqq.hqq_gated_linear_backward(*[torch.empty(3, 0, **bf)] * 3, w, w)[0] == 0).all()


# ------------------------------------------------------------------ streams, graphs, repetition

def block(seed=0, N=328, K=192, dtype="bf16"):
    gate, up = (Layer(N, K, 4, 64, 1, dtype, seed=seed + s) for s in (1, 2))
    down = Layer(K, N, 2, 8, 1, dtype, seed=seed + 3)
    return gate, up, down


def run_block(X, dOut, gate, up, down):
    """Forward and backward of a feed-forward block: every operator as they are used together."""
    Y, G, U = hqq.hqq_gated_linear(X, gate.h, up.h, save=True)
    out = hqq.hqq_linear_ex(Y, down.h)
    dY = hqq.hqq_linear_backward(dOut, down.h)
    dX, dG, dU = hqq.hqq_gated_linear_backward(dY, G, U, gate.h, up.h)
    return out, Y, G, U, dY, dX, dG, dU


@pytest.mark.parametrize("M", [1, 7, 70, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_feed_forward_block(M, dtype):
    """The chain, each step held to the formula on the inputs it was given, and the whole gradient
    to that of the block in 64 bits."""
    gate, up, down = block(dtype=dtype)
    X, X64 = draw((M, 192), 5, dtype, scale=0.05)
    dOut, dOut64 = draw((M, 192), 6, dtype, scale=0.1)
    out, Y, G, U, dY, dX, dG, dU = run_block(X, dOut, gate, up, down)
    S, e = down.project(host(Y))
    close(host(out), S, e, dtype, "out")
    e = 192 * 2.0 ** -23 * (np.abs(dOut64) @ np.abs(down.W))
    close(host(dY), dOut64 @ down.W, e, dtype, "dY")
    a, d = act64("silu", host(G))
    close(host(dU), host(dY) * a, np.abs(host(dY)) * (2 * ACT_REL["silu"] * np.abs(a) + 1e-12), dtype, "dU")
    # against the gradient of the 64-bit block: each rounded tensor on the way adds half a step to
    # each term of the sums behind it: G, U (act' <= 1.1, |act''| <= 0.5), dY, dG and dU
    g, u = X64 @ gate.W.T, X64 @ up.W.T
    a, d = act64("silu", g)
    dy = dOut64 @ down.W
    want = (dy * u * d) @ gate.W + (dy * a) @ up.W
    eps = UNIT[dtype]
    tg = np.abs(dy * u * d) * 3 * eps + np.abs(dy * u) * 0.5 * eps * np.abs(g)
    tu = np.abs(dy * a) * 2 * eps + np.abs(dy) * 1.1 * eps * np.abs(g)
    err = 1.05 * (tg @ np.abs(gate.W) + tu @ np.abs(up.W)) + \
        2 * 328 * 2.0 ** -23 * (np.abs(dy * u * d) @ np.abs(gate.W) + np.abs(dy * a) @ np.abs(up.W)) + \
        328 * TINY[dtype] * (np.abs(gate.W).max() + np.abs(up.W).max())
    close(host(dX), want, err, dtype, "dX of the block")


def test_gradient_against_differences():
    """dX of the block times a direction against central differences of the 64-bit block."""
    gate, up, down = block()
    X, X64 = draw((6, 192), 5, "bf16", scale=0.05)
    dOut, dOut64 = draw((6, 192), 6, "bf16", scale=0.1)
    dX = host(run_block(X, dOut, gate, up, down)[5])

    def loss(x):
        a, _ = act64("silu", x @ gate.W.T)
        return ((a * (x @ up.W.T)) @ down.W.T * dOut64).sum()

    rng = np.random.default_rng(0)
    for _ in range(4):
        v = rng.standard_normal(X64.shape)
        h = 1e-5
        want = (loss(X64 + h * v) - loss(X64 - h * v)) / (2 * h)
        # each element of dX is off by some four half steps of bf16 of its own size or of its row's
        # terms; in a random direction they add like a random walk: six of its standard deviations
        tol = 6 * 8 * UNIT["bf16"] * np.sqrt(((np.abs(dX) + np.abs(dX).mean()) ** 2 * v * v).sum())
        assert abs((dX * v).sum() - want) <= tol


@pytest.mark.parametrize("M", [4, 70, 300])
def test_other_streams(M):
    """A call on a side stream, with tensors of its own and given ones, gives the same bits."""
    gate, up, down = block()
    X, _ = draw((M, 192), 5, "bf16", scale=0.05)
    dOut, _ = draw((M, 192), 6, "bf16")
    want = run_block(X, dOut, gate, up, down)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y, G, U = hqq.hqq_gated_linear(X, gate.h, up.h, save=True, stream=side)
    out = hqq.hqq_linear_ex(Y, down.h, stream=side)
    dY = hqq.hqq_linear_backward(dOut, down.h, stream=side)
    dX, dG, dU = hqq.hqq_gated_linear_backward(dY, G, U, gate.h, up.h, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, (out, Y, G, U, dY, dX, dG, dU)):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        for a, b in zip(want, run_block(X, dOut, gate, up, down)):
            assert torch.equal(a, b)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [4, 70, 300])
def test_graph_replay_follows_its_inputs(M):
    gate, up, down = block()
    X, _ = draw((M, 192), 5, "bf16", scale=0.05)
    dOut, _ = draw((M, 192), 6, "bf16")
    run_block(X, dOut, gate, up, down)
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_block(X, dOut, gate, up, down))
        graphs.append(g)
    for seed in (7, 8):
        X.copy_(draw((M, 192), seed, "bf16", scale=0.05)[0])
        want = run_block(X, dOut, gate, up, down)
        for o in outs:
            for t in o:
                t.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(want, o):
                assert torch.equal(a, b)
    del graphs


def test_same_bits_every_time_and_with_a_given_workspace():
    for M, N, K in ((5, 1032, 4096), (100, 392, 4096), (300, 264, 2048)):
        L = Layer(N, K, 4, 64, 1, "bf16", seed=M)
        X, _ = draw((M, K), M, "bf16")
        first = hqq.hqq_linear_ex(X, L.h)
        ws = torch.full((hqq.hqq_linear_workspace_bytes(M, L.h),), 255, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            assert torch.equal(hqq.hqq_linear_ex(X, L.h), first)
            assert torch.equal(hqq.hqq_linear_ex(X, L.h, workspace=ws), first)
        X3 = X[:, None, :].contiguous()
        assert torch.equal(hqq.hqq_linear_ex(X3, L.h)[:, 0], first)


def test_two_calls_at_once():
    """Two streams, a workspace each, one weight."""
    L = Layer(520, 1024, 4, 64, 1, "bf16", seed=3)
    Xs = [draw((M, 1024), M, "bf16")[0] for M in (60, 90)]
    want = [hqq.hqq_linear_ex(X, L.h) for X in Xs]
    streams = [torch.cuda.Stream() for _ in Xs]
    torch.cuda.synchronize()
    outs = [[] for _ in Xs]
    for _ in range(20):
        for i, (X, s) in enumerate(zip(Xs, streams)):
            outs[i].append(hqq.hqq_linear_ex(X, L.h, stream=s))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, y) for y in o)


# ------------------------------------------------------------------ a weight beyond 2^32 codes

@pytest.mark.slow
@pytest.mark.parametrize("N,K", [(69632, 65600), (1100032, 4160)])
def test_more_than_2_pow_32_codes(N, K):
    """4 bits, group 64, 4.6e9 codes: code offsets pass 32 bits; checked on rows at the start, around
    code 2^32 and at the end. One token of the longer rows does not fit the few-token kernel, one
    of the shorter ones does."""
    G = 64
    g = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, generator=g, device="cuda")
    scale = (torch.rand(N * K // G, generator=g, device="cuda") * 0.01 + 1e-3).bfloat16()
    zero = (torch.rand(N * K // G, generator=g, device="cuda") * 15).bfloat16()
    prm = hqq.make_params(4, G, 1, w_dtype=torch.bfloat16)
    w = hqq.quantized_weight((packed, scale, zero), N, K, prm)
    cross = 2 ** 32 // K
    rows = torch.tensor([0, 1, cross - 1, cross, cross + 1, 2 * cross // 2 + 7, N - 9, N - 1], device="cuda")
    b = packed.view(N, K // 2)[rows]
    q = torch.stack([b & 15, b >> 4], -1).view(len(rows), K // G, G).float()
    s, z = scale.view(N, K // G)[rows].float(), zero.view(N, K // G)[rows].float()
    W = ((q - z[..., None]) * s[..., None]).bfloat16().double().view(len(rows), K)
    for M in (1, 9):
        X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        Y = hqq.hqq_linear_ex(X, w)[:, rows]
        want = X.double() @ W.T
        e = K * 2.0 ** -23 * (X.double().abs() @ W.abs().T)
        close(host(Y), want.cpu().numpy(), e.cpu().numpy(), "bf16", "Y")
    # the gradient of a row of dY that selects weight rows: their W', exactly
    dY = torch.zeros(len(rows), N, dtype=torch.bfloat16, device="cuda")
    dY[torch.arange(len(rows), device="cuda"), rows] = 1.0
    assert torch.equal(hqq.hqq_linear_backward(dY, w).double(), W)


@pytest.mark.parametrize("M", [1, 40, 600])
def test_a_weight_dropped_after_a_call_on_another_stream(M):
    """Its memory is not handed out again before that stream is done."""
    L = Layer(264, 320, 4, 64, 1, "bf16", bias=True, seed=M)
    X, _ = draw((M, 320), M, "bf16")
    want = hqq.hqq_linear_ex(X, L.h)
    torch.cuda.synchronize()
    pk, sc, zr, b = (t.clone() for t in L.h.tensors)
    sizes = [(t.shape, t.dtype) for t in (pk, sc, zr, b)]
    w = hqq.quantized_weight((pk, sc, zr), 264, 320, L.params, bias=b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    Y = hqq.hqq_linear_ex(X, w, stream=side)
    del w, pk, sc, zr, b
    for shape, dtype in sizes:
        torch.full(shape, 77, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


@pytest.mark.parametrize("nbits", NBITS)
def test_groups_of_16_on_odd_elements(nbits):
    """Scale and zero that cannot be loaded two groups at a time."""
    N, K = 72, 512
    L = Layer(N, K, nbits, 16, 1, "bf16", seed=nbits)

    def shifted(t):
        return torch.cat([t.new_zeros(1), t.reshape(-1)])[1:]

    pk, sc, zr = L.h.tensors[:3]
    w = hqq.quantized_weight((pk, shifted(sc), shifted(zr)), N, K, L.params)
    for M in (1, 8, 40):
        X, _ = draw((M, K), M, "bf16")
        dY, _ = draw((M, N), M, "bf16")
        assert torch.equal(hqq.hqq_linear_ex(X, w), hqq.hqq_linear_ex(X, L.h))
        assert torch.equal(hqq.hqq_gated_linear(X, w, L.h), hqq.hqq_gated_linear(X, L.h, L.h))
        assert torch.equal(hqq.hqq_linear_backward(dY, w), hqq.hqq_linear_backward(dY, L.h))


@pytest.mark.parametrize("M", [1, 8, 33])
@pytest.mark.parametrize("nbits,meta", [(2, "u8"), (3, "u8scale"), (4, "f32"), (8, "u8zero"), (1, "f16")])
def test_gated_in_groups_of_16_with_other_meta(nbits, meta, M):
    N, K = 136, 512
    gate, up = (Layer(N, K, nbits, 16, 1, "bf16", meta, seed=nbits + i) for i in (0, 50))
    X, X64 = draw((M, K), M, "bf16", scale=0.02)
    check_gated(M, N, K, "silu", "bf16", gate, up, X, X64)


# ------------------------------------------------------------------ many tiles for every CTA pair

def in_parts(call, *tensors, rows=4096):
    """The call on blocks of the tokens, one after the other: its outputs, joined."""
    parts = [call(*(t[m:m + rows].contiguous() for t in tensors)) for m in range(0, len(tensors[0]), rows)]
    return [torch.cat(p) for p in zip(*parts)]


def close_on_device(got, A, W, L, dtype, what):
    """Every element of got = A W^T in 64 bits, on the GPU."""
    A, W = A.double(), torch.from_numpy(W).cuda()
    want, u = A @ W.T, UNIT[dtype]
    tol = u * want.abs() + (1 + u) * L * 2.0 ** -23 * (A.abs() @ W.abs().T) + TINY[dtype]
    assert ((got.double() - want).abs() <= tol).all(), what


@pytest.mark.parametrize("N", [1056, 2312, 2784])
@pytest.mark.parametrize("K", [64, 256])
def test_every_row_of_many_tiles_with_a_ragged_last_column(N, K):
    """32 row blocks of 256 tokens: a CTA pair goes on from a tile that N cuts off after an odd number of
    32-column blocks to others, with so short a contraction that nothing else holds it up. Bit for bit
    what calls of 4096 tokens give, where no pair does."""
    M, G = 8192, 8 if N % 32 else 32
    X, _ = draw((M, K), 1, "bf16", scale=0.3)
    L, up = (Layer(N, K, 4, 64, 1, "bf16", seed=s) for s in (K, K + 1))
    back = Layer(K, N, 4, G, 1, "bf16", seed=N)  # dX has N columns
    for _ in range(3):
        Y = hqq.hqq_linear_ex(X, L.h)
        assert torch.equal(Y, in_parts(lambda x: (hqq.hqq_linear_ex(x, L.h),), X)[0])
        dX = hqq.hqq_linear_backward(X, back.h)
        assert torch.equal(dX, in_parts(lambda x: (hqq.hqq_linear_backward(x, back.h),), X)[0])
        pair = hqq.hqq_gated_linear(X, L.h, up.h, save=True)
        for a, b in zip(pair, in_parts(lambda x: hqq.hqq_gated_linear(x, L.h, up.h, save=True), X)):
            assert torch.equal(a, b)
    close_on_device(Y, X, L.W, K, "bf16", "Y")
    close_on_device(dX, X, back.W.T.copy(), K, "bf16", "dX")
    close_on_device(pair[1], X, L.W, K, "bf16", "G")
    close_on_device(pair[2], X, up.W, K, "bf16", "U")


# ------------------------------------------------------------------ host threads

@pytest.mark.parametrize("sizes", [((8, 1024), (1, 512)), ((16, 1024), (200, 1024))])
def test_two_host_threads_at_different_sizes(sizes):
    """Calls of one kernel that want different amounts of shared memory, from two threads at once."""
    layers = {K: Layer(136, K, 4, 64, 1, "bf16", seed=K) for _, K in sizes}
    failed = []

    def work(M, K):
        try:
            X, _ = draw((M, K), M, "bf16")
            stream = torch.cuda.Stream()
            want = hqq.hqq_linear_ex(X, layers[K].h)
            Y, n = torch.empty_like(want), hqq.hqq_linear_workspace_bytes(M, layers[K].h)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
            torch.cuda.synchronize()
            args = (X.data_ptr(), M, hqq.HQQ_BF16, layers[K].h.ptr, Y.data_ptr(), ws.data_ptr() if n else None,
                    n, stream.cuda_stream)
            call = hqq.lib().hqq_linear_ex  # without the interpreter lock
            for _ in range(20000):
                assert call(*args) == 0
            stream.synchronize()
            assert torch.equal(Y, want)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=s) for s in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("nbits", NBITS)
def test_one_hot_with_zeros_beyond_the_reach_of_a_sum(nbits):
    """Zeros of 2^20 to 2^40 whose products with the scale are ties of bf16: one step of fp32 in
    code - zero turns W' over."""
    N, K, G = 64, 4096, 64
    rng = np.random.default_rng(nbits)
    z, s = np.meshgrid(np.arange(128, 256), np.arange(128, 256), indexing="ij")
    p = z * s
    tie = np.where(p < 1 << 15, p % 128 == 64, p % 256 == 128)
    pick = rng.integers(0, tie.sum(), N * K // G)
    e = rng.integers(20 - 7, 41 - 7, pick.size)
    zero = (z[tie][pick] * 2.0 ** e * rng.choice([-1.0, 1.0], pick.size)).astype(np.float32)
    scale = (s[tie][pick] * 2.0 ** (-7 - e)).astype(np.float32)
    codes = rng.integers(0, 2 ** nbits, size=N * K, dtype=np.uint8)
    W = oracle.round_to_dtype(oracle.dequantize(codes, scale, zero, N, K, G, 1), "bf16")
    q = [torch.from_numpy(oracle.pack(codes, nbits)).cuda()] + \
        [torch.from_numpy(v).bfloat16().cuda() for v in (scale, zero)]
    assert all(np.array_equal(host(t), v) for t, v in zip(q[1:], (scale, zero)))
    w = hqq.quantized_weight(q, N, K, hqq.make_params(nbits, G, 1, w_dtype=torch.bfloat16))
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    for n in (8, 64):
        for k0 in range(0, K, n):
            assert np.array_equal(host(hqq.hqq_linear_ex(eye[k0:k0 + n], w)), W.T[k0:k0 + n])
    eye = torch.eye(N, dtype=torch.bfloat16, device="cuda")
    assert np.array_equal(host(hqq.hqq_linear_backward(eye, w)), W)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_derivatives_far_out(act):
    """Gates so far out that act' is 1 or 0 to more than 64 bits, up to the largest of bf16."""
    L = Layer(64, 64, 4, 64, 1, "bf16", seed=1)
    g = torch.tensor([1e3, 1e9, 1e18, 2e19, 1e20, 1e30, 3e38, torch.finfo(torch.bfloat16).max] * 8,
                     device="cuda").bfloat16().repeat(2, 1)
    g[1] *= -1
    dY, _ = draw((2, 64), 1, "bf16", scale=1e-3)
    u, _ = draw((2, 64), 2, "bf16")
    dX, dG, dU = hqq.hqq_gated_linear_backward(dY, g, u, L.h, L.h, act)
    want = (dY.double() * u.double())
    assert ((dG[0].double() - want[0]).abs() <= 2.0 ** -8 * (1 + 2.0 ** -15) * want[0].abs()).all()
    assert (dG[1] == 0).all() and (dU[1] == 0).all()
    assert torch.isfinite(dU).all() and torch.isfinite(dX).all()


# ------------------------------------------------------------------ autograd

def test_an_input_that_requires_a_gradient_is_not_dropped_silently():
    L = Layer(64, 128, 4, 64, 1, "bf16", seed=1)
    X, _ = draw((3, 128), 1, "bf16")
    want = hqq.hqq_linear_ex(X, L.h)
    calls = (lambda x: hqq.hqq_linear_ex(x, L.h), lambda x: hqq.hqq_gated_linear(x, L.h, L.h))
    for call in calls:
        with pytest.warns(UserWarning, match="no gradient"):
            call(X.clone().requires_grad_())
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for call in calls:
            call(X)
            with torch.no_grad():
                call(X.clone().requires_grad_())

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, w):
            ctx.w = w
            return hqq.hqq_linear_ex(X, w)

        @staticmethod
        def backward(ctx, dY):
            return hqq.hqq_linear_backward(dY.contiguous(), ctx.w), None

    leaf = X.clone().requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Y = Linear.apply(leaf, L.h)
        assert torch.equal(Y, want)
        dY, _ = draw((3, 64), 2, "bf16")
        Y.backward(dY)
    assert torch.equal(leaf.grad, hqq.hqq_linear_backward(dY, L.h))
