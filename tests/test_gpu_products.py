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
