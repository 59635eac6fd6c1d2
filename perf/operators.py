"""The products of layers over quantized weights: what is measured of them, and their plain forms.

Four operators over weights as the quantizer packs them (any code width, group size, axis and
meta type): a linear layer for every format (``hqq_linear_ex``), its gradient
(``hqq_linear_backward``), and the gated pair of projections of a feed-forward block
(``hqq_gated_linear``) with its gradient (``hqq_gated_linear_backward``).

Throughout, W' is the weight that dequantization writes: (code - zero) * scale in fp32, rounded
once to the activations' type. That rounding belongs to the operators' definition (a quantized
layer computes in its compute type from the dequantized weight), and so does that of dG and dU,
which the gated gradient returns and multiplies. All other rounding is of the outputs alone.

    linear            Y  = X W'^T + bias
    linear gradient   dX = dY W',  dbias = column sums of dY
    gated             G  = X Wg'^T + bg,  U = X Wu'^T + bu,  Y = act(G) * U   (G, U unrounded)
    gated gradient    dG = dY * U * act'(G),  dU = dY * act(G)   (from the saved, rounded G, U)
                      dX = dG Wg' + dU Wu',  dbg, dbu = column sums of dG, dU
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# The largest product and the largest weight that a case may have (the largest listed ones).
_MOST_MACS = 2 * 4096 * 11008 * 4096
_MOST_WEIGHTS = 28672 * 8192


def _case(name, op, M, N, K, nbits, G, axis=1, dtype="bf16", meta="same", act="silu", bias=False,
          save=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "nbits": nbits, "G": G, "axis": axis,
            "dtype": dtype, "meta": meta, "act": act, "bias": bias, "save": save}


def listed():
    return [
        # one token through the small fp16 layer: the smallest call, where latency counts
        _case("linear_1tok_4096x1024_4b", "linear", 1, 4096, 1024, 4, 64, dtype="fp16"),
        # one token through a 7B-class MLP projection: ordinary decoding
        _case("linear_1tok_11008x4096_4b", "linear", 1, 11008, 4096, 4, 64),
        # a few tokens through a 70B-class MLP weight at 3 bits with 8-bit scale and zero
        _case("linear_5tok_28672x8192_3b_meta8", "linear", 5, 28672, 8192, 3, 64, meta="u8"),
        # a decode batch through a first-block projection at 8 bits, group 128, with bias
        _case("linear_16tok_4096x11008_8b", "linear", 16, 4096, 11008, 8, 128, bias=True),
        # a ragged prompt through the 2-bit group-16 down projection of the mixed model
        _case("linear_333tok_4096x11008_2b", "linear", 333, 4096, 11008, 2, 16),
        # one token through the gate and up projections
        _case("gated_1tok_11008x4096_4b", "gated", 1, 11008, 4096, 4, 64),
        # an odd decode batch through the 2-bit group-16 gate and up of the mixed model
        _case("gated_37tok_11008x4096_2b", "gated", 37, 11008, 4096, 2, 16),
        # a training step's forward pass: 4096 tokens, G and U kept for the gradient
        _case("gated_4096tok_11008x4096_4b", "gated", 4096, 11008, 4096, 4, 64, save=True),
        # a training step's gradient through the frozen down projection
        _case("linear_grad_4096tok_4096x11008_4b", "linear_grad", 4096, 4096, 11008, 4, 64),
        # the gradient of a short fp16 batch through a 1-bit group-32 weight with 8-bit meta
        _case("linear_grad_77tok_28672x8192_1b", "linear_grad", 77, 28672, 8192, 1, 32,
              dtype="fp16", meta="u8", bias=True),
        # a training step's gradient through the gated pair
        _case("gated_grad_4096tok_11008x4096_4b", "gated_grad", 4096, 11008, 4096, 4, 64),
        # the gradient of an odd batch, groups down the columns, fp32 meta, biases, gelu
        _case("gated_grad_129tok_11008x4096_2b_axis0", "gated_grad", 129, 11008, 4096, 2, 16,
              axis=0, meta="fp32", act="gelu", bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "linear_grad", "gated_grad"])
    mats = 2 if op.startswith("gated") else 1
    axis = 1 if rng.random() < 0.8 else 0
    nbits = rng.choice([8, 4, 4, 4, 3, 2, 1])
    G = rng.choice([8, 16, 32, 64, 64, 64, 128, 256])
    # half of the forward calls are decode batches, the others prompts of any length
    forward = not op.endswith("grad")
    M = _log_int(rng, 1, 64) if forward and rng.random() < 0.5 else _log_int(rng, 1, 4096)
    kstep, nstep = (G, 8) if axis == 1 else (8, max(G, 8))
    K = max(1, _log_int(rng, 256, 12288) // kstep) * kstep
    N = max(1, _log_int(rng, 256, 28672) // nstep) * nstep
    while mats * N * K > _MOST_WEIGHTS:
        N = max(1, N // 2 // nstep) * nstep
    M = max(1, min(M, _MOST_MACS // (mats * N * K)))
    return {"op": op, "M": M, "N": N, "K": K, "nbits": nbits, "G": G, "axis": axis,
            "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "meta": rng.choice(["same", "same", "fp32", "u8"]),
            "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
            "bias": rng.random() < 0.3, "save": op == "gated" and rng.random() < 0.4}


# ------------------------------------------------------------------------------ inputs

def _pack(codes, nbits):
    """The packed stream of uint8 codes: least significant code first in each byte; 3-bit codes
    ten to a 32-bit word."""
    if nbits == 8:
        return codes
    if nbits == 3:
        c = torch.nn.functional.pad(codes, (0, -codes.numel() % 10)).view(-1, 10).to(torch.int32)
        shift = torch.arange(0, 30, 3, dtype=torch.int32, device=codes.device)
        return (c << shift).sum(1, dtype=torch.int32).view(torch.uint8)
    per = 8 // nbits
    c = codes.view(-1, per)
    out = c[:, 0].clone()
    for i in range(1, per):
        out |= c[:, i] << (nbits * i)
    return out


def _meta8(v, run=128):
    """8-bit round-to-nearest of v in runs of 128 values: codes, (step, zero) pairs."""
    n = v.numel()
    p = torch.cat([v, v[-1:].expand(-n % run)]).view(-1, run)
    lo, hi = p.amin(1, keepdim=True), p.amax(1, keepdim=True)
    same = hi == lo
    step = torch.where(same, torch.ones_like(hi), (hi - lo) / 255)
    inv = torch.where(same, torch.ones_like(hi), 255 / (hi - lo))
    z = -lo * inv
    q = (p * inv + z).round_().clamp_(0, 255).to(torch.uint8)
    return q.view(-1)[:n].contiguous(), torch.cat([step, z], 1).contiguous()


def _weight(case, g, bias):
    """A quantized [N, K] weight: gaussian weights of a layer (sigma 0.02, a few outliers),
    rounded to nearest per group, as a quantized checkpoint holds them."""
    N, K, G, axis, nbits = case["N"], case["K"], case["G"], case["axis"], case["nbits"]
    shape = (N, K // G, G) if axis == 1 else (N // G, K, G)  # groups in stream order
    w = torch.randn(shape, generator=g, device="cuda").mul_(0.02)
    rows = torch.randn((shape[0], 1, 1), generator=g, device="cuda").mul_(0.3).exp_()
    w.mul_(rows)
    w[:, :, 0] *= torch.where(torch.rand(shape[:2], generator=g, device="cuda") < 0.01, 6.0, 1.0)
    qmax = 2 ** nbits - 1
    lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
    step = (hi - lo) / qmax
    zero = -lo / step
    codes = (w / step + zero).round_().clamp_(0, qmax).to(torch.uint8).view(-1)
    packed = _pack(codes, nbits)
    q = {"Wq_packed": packed, "scale_mm": None, "zero_mm": None}
    if case["meta"] == "u8":
        q["scale"], q["scale_mm"] = _meta8(step.reshape(-1))
        q["zero"], q["zero_mm"] = _meta8(zero.reshape(-1))
    else:
        dt = _DT[case["dtype"] if case["meta"] == "same" else "fp32"]
        q["scale"] = step.reshape(-1).to(dt)
        q["zero"] = zero.reshape(-1).to(dt)
    meta_shape = (N, K // G) if axis == 1 else (N // G, K)
    q["scale"], q["zero"] = q["scale"].view(meta_shape), q["zero"].view(meta_shape)
    q["bias"] = torch.randn(N, generator=g, device="cuda").mul_(0.1).to(_DT[case["dtype"]]) \
        if bias else None
    return q


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, M, N, K = _DT[case["dtype"]], case["M"], case["N"], case["K"]
    op = case["op"]
    mats = 2 if op.startswith("gated") else 1
    s = {"case": dict(case), "w": [_weight(case, g, case["bias"]) for _ in range(mats)]}

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dt)

    if op in ("linear", "gated"):
        s["X"] = normal(M, K)  # normalised hidden states
    else:
        s["dY"] = normal(M, N, scale=0.01)
    if op == "gated_grad":
        s["G"], s["U"] = normal(M, N, scale=1.3), normal(M, N, scale=1.3)
    if own:  # what a program that holds the layer keeps: its weights' handles
        import calibration_free_weight_hqq_b200 as hqq
        prm = hqq.make_params(case["nbits"], case["G"], case["axis"], w_dtype=dt,
                              meta_dtype=torch.float32 if case["meta"] == "fp32" else dt,
                              quant_scale=case["meta"] == "u8", quant_zero=case["meta"] == "u8")
        s["handles"] = [hqq.quantized_weight(w, N, K, prm, bias=w["bias"]) for w in s["w"]]
    return s


# --------------------------------------------------------------------------- plain forms

def _unpack(packed, nbits, n):
    if nbits == 8:
        return packed
    if nbits == 3:
        shift = torch.arange(0, 30, 3, dtype=torch.int32, device=packed.device)
        return ((packed.view(torch.int32)[:, None] >> shift) & 7).view(-1)[:n]
    shift = torch.arange(0, 8, nbits, dtype=torch.uint8, device=packed.device)
    return ((packed[:, None] >> shift) & (2 ** nbits - 1)).view(-1)


def _meta_plain(v, mm):
    """Scale or zero in fp32: (code - zero2) * step2 of its run where it is held in 8 bits."""
    v = v.reshape(-1).float()
    if mm is None:
        return v
    pair = mm.repeat_interleave(128, 0)[:v.numel()]
    return (v - pair[:, 1]) * pair[:, 0]


def _dequantized(case, w):
    """W' [N, K] in fp32, holding values of the activations' type (see the module's text)."""
    N, K, G, axis = case["N"], case["K"], case["G"], case["axis"]
    q = _unpack(w["Wq_packed"], case["nbits"], N * K).view(-1, G).float()
    v = (q - _meta_plain(w["zero"], w["zero_mm"])[:, None]) * \
        _meta_plain(w["scale"], w["scale_mm"])[:, None]
    v = v.view(N, K) if axis == 1 else v.view(N // G, K, G).permute(0, 2, 1).reshape(N, K)
    return v.to(_DT[case["dtype"]]).float()


_C = math.sqrt(2 / math.pi)


def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(_C * (g + 0.044715 * g * g * g)))


def _act_grad(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + \
            g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _C * (1 + 3 * 0.044715 * g * g)


def _project(case, X, w):
    y = X @ _dequantized(case, w).T
    return y if w["bias"] is None else y + w["bias"].float()


def _run_plain(s):
    case, w = s["case"], s["w"]
    dt, op = _DT[case["dtype"]], case["op"]
    if op == "linear":
        return {"Y": _project(case, s["X"].float(), w[0]).to(dt)}
    if op == "gated":
        X = s["X"].float()
        g, u = _project(case, X, w[0]), _project(case, X, w[1])
        out = {"Y": (_act(case["act"], g) * u).to(dt)}
        return {**out, "G": g.to(dt), "U": u.to(dt)} if case["save"] else out
    dY = s["dY"].float()
    if op == "linear_grad":
        out = {"dX": (dY @ _dequantized(case, w[0])).to(dt)}
        return {**out, "dbias": dY.sum(0).to(dt)} if case["bias"] else out
    g, u = s["G"].float(), s["U"].float()
    dG = (dY * u * _act_grad(case["act"], g)).to(dt)
    dU = (dY * _act(case["act"], g)).to(dt)
    dX = dG.float() @ _dequantized(case, w[0]) + dU.float() @ _dequantized(case, w[1])
    out = {"dX": dX.to(dt), "dG": dG, "dU": dU}
    if case["bias"]:
        out.update(dbg=dG.float().sum(0).to(dt), dbu=dU.float().sum(0).to(dt))
    return out


def _run_own(s):
    import calibration_free_weight_hqq_b200 as hqq
    case, h = s["case"], s["handles"]
    op = case["op"]
    if op == "linear":
        return {"Y": hqq.hqq_linear_ex(s["X"], h[0])}
    if op == "gated":
        if not case["save"]:
            return {"Y": hqq.hqq_gated_linear(s["X"], h[0], h[1], case["act"])}
        Y, G, U = hqq.hqq_gated_linear(s["X"], h[0], h[1], case["act"], save=True)
        return {"Y": Y, "G": G, "U": U}
    if op == "linear_grad":
        if not case["bias"]:
            return {"dX": hqq.hqq_linear_backward(s["dY"], h[0])}
        dX, db = hqq.hqq_linear_backward(s["dY"], h[0], bias_grad=True)
        return {"dX": dX, "dbias": db}
    got = hqq.hqq_gated_linear_backward(s["dY"], s["G"], s["U"], h[0], h[1], case["act"],
                                        bias_grad=case["bias"])
    return dict(zip(("dX", "dG", "dU", "dbg", "dbu"), got))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------- work and values

def work(case):
    M, N, K, G, op = case["M"], case["N"], case["K"], case["G"], case["op"]
    mats = 2 if op.startswith("gated") else 1
    groups = N * K // G
    per_meta = 1 + 8 / 128 if case["meta"] == "u8" else 4 if case["meta"] == "fp32" else 2
    code = 4 * ((N * K + 9) // 10) if case["nbits"] == 3 else N * K * case["nbits"] / 8
    nbytes = mats * (code + 2 * groups * per_meta)
    if op == "linear":
        nbytes += 2 * M * (K + N)
    elif op == "gated":
        nbytes += 2 * M * (K + N) + (4 * M * N if case["save"] else 0)
    elif op == "linear_grad":
        nbytes += 2 * M * (K + N)
    else:
        nbytes += 2 * M * (K + 5 * N)
    if case["bias"]:
        nbytes += 2 * N * mats
    return {"bytes": nbytes, "flops": 2 * M * N * K * mats}


def _exact_weight(case, w):
    """W' [N, K]: the values dequantization writes (fp32 arithmetic, one rounding to the
    activations' type, as defined), held in 64 bits. Each element's code is looked up by its
    place in the stream."""
    N, K, G, axis, b = case["N"], case["K"], case["G"], case["axis"], case["nbits"]
    out = torch.empty(N, K, dtype=torch.float64, device="cuda")
    col = torch.arange(K, device="cuda")[None, :]
    step = max(G, (1 << 25) // K // G * G)
    scale, zero = w["scale"].reshape(-1), w["zero"].reshape(-1)
    for r0 in range(0, N, step):
        row = torch.arange(r0, min(N, r0 + step), device="cuda")[:, None]
        group = row * (K // G) + col // G if axis == 1 else row // G * K + col
        place = group * G + (col % G if axis == 1 else row % G)
        if b == 3:
            code = w["Wq_packed"].view(torch.int32)[place // 10] >> (place % 10 * 3).int()
        else:
            code = w["Wq_packed"][place * b // 8].int() >> (place * b % 8).int()
        code = (code & (2 ** b - 1)).float()
        s, z = scale[group].float(), zero[group].float()
        if w["scale_mm"] is not None:
            s = (s - w["scale_mm"][group // 128, 1]) * w["scale_mm"][group // 128, 0]
            z = (z - w["zero_mm"][group // 128, 1]) * w["zero_mm"][group // 128, 0]
        out[r0:r0 + step] = ((code - z) * s).to(_DT[case["dtype"]]).double()
    return out


def _exact_act(name, g):
    """act(g) and its derivative in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * inner)  # (1 + tanh(inner)) / 2
    return g * s, s + g * 2 * s * (1 - s) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, dt = case["op"], _DT[case["dtype"]]
    W = [_exact_weight(case, w) for w in s["w"]]
    b = [0.0 if w["bias"] is None else w["bias"].double() for w in s["w"]]
    if op == "linear":
        return {"Y": s["X"].double() @ W[0].T + b[0]}
    if op == "gated":
        X = s["X"].double()
        g, u = X @ W[0].T + b[0], X @ W[1].T + b[1]
        out = {"Y": _exact_act(case["act"], g)[0] * u}
        return {**out, "G": g, "U": u} if case["save"] else out
    dY = s["dY"].double()
    if op == "linear_grad":
        out = {"dX": dY @ W[0]}
        return {**out, "dbias": dY.sum(0)} if case["bias"] else out
    a, d = _exact_act(case["act"], s["G"].double())
    dG, dU = dY * s["U"].double() * d, dY * a
    rG, rU = dG.to(dt).double(), dU.to(dt).double()  # what is written is what is multiplied
    out = {"dX": rG @ W[0] + rU @ W[1], "dG": dG, "dU": dU}
    if case["bias"]:
        out.update(dbg=rG.sum(0), dbu=rU.sum(0))
    return out
