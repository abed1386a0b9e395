"""Measured cases of the pointwise feed-forward in 8-bit integers.

A token is one pixel of one sample; activations are [B, C, P], and P = 1 is the
layout of rows of features.

Linear layer (``disco_quant_i8`` and ``disco_matmul_i8``): every token in 8-bit
integers with a scale of its own, then the product with a weight in 8-bit
integers with a scale for each output channel.  Its gradients
(``disco_matmul_i8_bwd_input``, ``disco_matmul_i8_bwd_weight``) need the 8-bit
activation alone, which a training program keeps in place of the 16-bit one.

Gated activation (``disco_glu``): act(gate) * value, in 8 bits for the layer
that follows, or with its input kept in 8 bits for ``disco_glu_bwd``.

``run`` computes a pass in plain torch operations in 32 bits, or with ``own``
by the library; ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

Q_MAX = 127.0
AMAX_FLOOR = 1e-30
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
ACTS = ("silu", "gelu")


def _linear(name, B, Cin, Cout, P, dtype):
    return {"name": name, "op": "linear", "B": B, "Cin": Cin, "Cout": Cout, "P": P, "dtype": dtype}


def _bwd(name, B, Cin, Cout, P, dtype):
    return {"name": name, "op": "linear_bwd", "B": B, "Cin": Cin, "Cout": Cout, "P": P, "dtype": dtype}


def _glu_down(name, B, C, Cout, P, dtype, act):
    return {"name": name, "op": "glu_down", "B": B, "Cin": C, "Cout": Cout, "P": P, "dtype": dtype, "act": act}


def _glu_train(name, B, C, P, dtype, act):
    return {"name": name, "op": "glu_train", "B": B, "Cin": C, "Cout": 0, "P": P, "dtype": dtype, "act": act}


def listed():
    return [
        # one pooled feature vector widened in a head: the latency of a call
        _linear("linear 1x512->2048", 1, 512, 2048, 1, "bf16"),
        # a batch of feature vectors through a head
        _linear("linear rows 96x2048->2048", 96, 2048, 2048, 1, "bf16"),
        # a pointwise layer at the library's 512-channel shape on the 360 x 720 grid
        _linear("linear 512->512 360x720", 1, 512, 512, 360 * 720, "bf16"),
        # an odd grid with odd channel counts: no row but the first is aligned
        _linear("linear odd 3x80->77 181x361", 3, 80, 77, 181 * 361, "f16"),
        # per-pixel features gathered into rows (a point head)
        _linear("linear rows 16384x2048->2048", 16384, 2048, 2048, 1, "bf16"),
        # gradients of a pointwise layer from the 8-bit activation: a small odd grid, a large grid, rows
        _bwd("bwd 4x64->48 33x65", 4, 64, 48, 33 * 65, "f16"),
        _bwd("bwd 2x128->256 361x720", 2, 128, 256, 361 * 720, "bf16"),
        _bwd("bwd rows 16384x2048->2048", 16384, 2048, 2048, 1, "bf16"),
        # the second half of a gated feed-forward: a few feature vectors, a grid
        _glu_down("glu+down rows 8x2048->512", 8, 2048, 512, 1, "bf16", "silu"),
        _glu_down("glu+down 2x256->128 361x720", 2, 256, 128, 361 * 720, "bf16", "silu"),
        # the gated activation in training, its input kept in 8 bits: a grid, and rows of an odd length in 32 bits
        _glu_train("glu train 2x128 361x720", 2, 128, 361 * 720, "bf16", "silu"),
        _glu_train("glu train rows 4099x1365", 4099, 1365, 1, "f32", "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "glu_down", "glu_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "linear_bwd" and dtype == "f32":
        dtype = "f16"
    if rng.random() < 0.5:  # rows
        P, B = 1, _log(rng, 1, 32768)
        cin, cout = _log(rng, 16, 8192), _log(rng, 16, 8192)
    else:
        nlat = _log(rng, 4, 721)
        P = nlat * (2 * nlat if rng.random() < 0.6 else nlat + rng.randint(0, 2 * nlat))
        B, cin, cout = _log(rng, 1, 16), _log(rng, 3, 768), _log(rng, 3, 768)
    if rng.random() < 0.5:  # channel counts of real layers are mostly round
        cin, cout = -(-cin // 16) * 16, -(-cout // 16) * 16
    wide = 2 if op.startswith("glu") else 1
    while B * P * max(wide * cin, cout) > 60_000_000 or (op != "glu_train" and B * P * cin * cout > 50_000_000_000):
        if B > 1:
            B = B // 2
        else:
            cin, cout = (cin + 1) // 2, (cout + 1) // 2
    c = {"op": op, "B": B, "Cin": cin, "Cout": cout if op != "glu_train" else 0, "P": P, "dtype": dtype}
    if op.startswith("glu"):
        c["act"] = rng.choice(ACTS)
    return c


# ------------------------------------------------------------------ inputs

def _quant(x):
    """(q, scale) of the tokens of x [B, C, P], in 32 bits.  127 x is exact for 16-bit types, and the quotient's
    rounding then moves no value over a border; next to one, 32-bit inputs need 64 bits."""
    x = x.float() if x.dtype != torch.float32 else x.double()
    amax = x.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
    return torch.round(x * Q_MAX / amax).to(torch.int8), (amax / Q_MAX).float()[:, 0]


def _inputs(case, seed):
    """The tensors of a case, made on the GPU from the seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    B, Cin, Cout, P, dt = case["B"], case["Cin"], case["Cout"], case["P"], DTYPES[case["dtype"]]
    s = {}
    if Cout:
        # output channels of a trained weight differ in size
        w = randn(Cout, Cin) * (0.5 + torch.rand((Cout, 1), generator=g, device="cuda")) / math.sqrt(Cin)
        s["W"], s["wscale"] = _quant(w.view(Cout, Cin, 1))
        s["W"], s["wscale"] = s["W"].view(Cout, Cin), s["wscale"].view(Cout)
    if case["op"].startswith("glu"):
        s["x"] = randn(B, 2 * Cin, P).mul_(1.5).to(dt)
        if case["op"] == "glu_train":
            s["dy"] = (1e-2 * randn(B, Cin, P)).to(dt)
        return s
    # after a norm: unit size, some channels several times the others
    x = (randn(B, Cin, P) * (0.5 + 2 * torch.rand((Cin, 1), generator=g, device="cuda") ** 4)).to(dt)
    if case["op"] == "linear":
        s["x"] = x
    else:
        s["q"], s["scale"] = _quant(x)
        s["dy"] = (1e-2 * randn(B, Cout, P)).to(dt)
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    # what the program owns: output and 8-bit buffers, and for the library's calls their workspace
    B, Cin, Cout, P, dt = case["B"], case["Cin"], case["Cout"], case["P"], DTYPES[case["dtype"]]

    def new(C, d=dt):
        return torch.empty((B, C, P), dtype=d, device="cuda")

    if case["op"] in ("linear", "glu_down"):
        s["q"], s["scale"], s["y"] = new(Cin, torch.int8), torch.empty((B, P), device="cuda"), new(Cout)
    elif case["op"] == "linear_bwd":
        s["dx"], s["dW"] = new(Cin), torch.empty((Cout, Cin), dtype=dt, device="cuda")
    else:
        s["y"], s["dx"] = new(Cin), new(2 * Cin)
        s["xq"], s["xscale"] = new(2 * Cin, torch.int8), torch.empty((B, P), device="cuda")
    if own and Cout:
        import sparse_spherical_convolution_gb300 as d
        code = d.dtype_code(dt)
        sizes = ([d.disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, code)] if case["op"] != "linear_bwd" else
                 [d.disco_matmul_i8_bwd_input_workspace_bytes(B, Cin, Cout, P, code),
                  d.disco_matmul_i8_bwd_weight_workspace_bytes(B, Cin, Cout, P, code)])
        s["workspace"] = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    cdf = 0.5 * torch.erfc(-g * math.sqrt(0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _product(q, scale, W, wscale):
    y = torch.matmul(W.float(), q.float()) if q.shape[2] > 1 else torch.matmul(q[:, :, 0].float(), W.float().t())[:, :, None]
    return y * (wscale[:, None] * scale[:, None])


def run(s):
    case = s["case"]
    if own:
        return _run_library(s, case)
    dt, C = DTYPES[case["dtype"]], case["Cin"]
    if case["op"] == "linear":
        return {"y": _product(*_quant(s["x"]), s["W"], s["wscale"]).to(dt)}
    if case["op"] == "linear_bwd":
        dy, x = s["dy"].float(), s["q"].float() * s["scale"][:, None]
        W = s["W"].float() * s["wscale"][:, None]
        if case["P"] == 1:
            dx, dW = torch.matmul(dy[:, :, 0], W)[:, :, None], torch.matmul(dy[:, :, 0].t(), x[:, :, 0])
        else:
            dx, dW = torch.matmul(W.t(), dy), torch.matmul(dy, x.transpose(1, 2)).sum(0)
        return {"dx": dx.to(dt), "dW": dW.to(dt)}
    x = s["x"].float()
    y = _act(x[:, :C], case["act"])[0] * x[:, C:]
    if case["op"] == "glu_down":
        amax = y.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
        return {"y": _product(torch.round(y * Q_MAX / amax), (amax / Q_MAX)[:, 0], s["W"], s["wscale"]).to(dt)}
    q, scale = _quant(s["x"])
    kept, dy = q.float() * scale[:, None], s["dy"].float()
    a, da = _act(kept[:, :C], case["act"])
    return {"y": y.to(dt), "dx": torch.cat([dy * kept[:, C:] * da, dy * a], 1).to(dt)}


def _run_library(s, case):
    import sparse_spherical_convolution_gb300 as d
    B, Cin, Cout, P = case["B"], case["Cin"], case["Cout"], case["P"]
    if case["op"] == "linear_bwd":
        d.disco_matmul_i8_bwd_input(s["dy"], s["W"], s["wscale"], s["dx"], B, Cin, Cout, P, s["workspace"])
        d.disco_matmul_i8_bwd_weight(s["dy"], s["q"], s["scale"], s["dW"], B, Cin, Cout, P, s["workspace"])
        return {"dx": s["dx"], "dW": s["dW"]}
    if case["op"] == "glu_train":
        act = d.DISCO_SILU if case["act"] == "silu" else d.DISCO_GELU
        d.disco_glu(s["x"], s["y"], act, B, Cin, P, xq=s["xq"], xscale=s["xscale"])
        d.disco_glu_bwd(s["dy"], s["xq"], s["xscale"], s["dx"], act, B, Cin, P)
        return {"y": s["y"], "dx": s["dx"]}
    if case["op"] == "linear":
        d.disco_quant_i8(s["x"], s["q"], s["scale"], B, Cin, P)
    else:
        act = d.DISCO_SILU if case["act"] == "silu" else d.DISCO_GELU
        d.disco_glu(s["x"], None, act, B, Cin, P, q=s["q"], scale=s["scale"])
    d.disco_matmul_i8(s["q"], s["scale"], s["W"], s["wscale"], s["y"], B, Cin, Cout, P, s["workspace"])
    return {"y": s["y"]}


def work(case):
    B, Cin, Cout, P, e = case["B"], case["Cin"], case["Cout"], case["P"], SIZES[case["dtype"]]
    T = B * P
    weight = Cout * Cin + 4 * Cout
    if case["op"] == "linear":
        return {"bytes": T * e * (Cin + Cout) + weight, "flops": 2 * T * Cin * Cout + 3 * T * Cin}
    if case["op"] == "linear_bwd":
        # dy once for both gradients, the 8-bit activation and its scales, both gradients
        return {"bytes": T * (e * (Cin + Cout) + Cin + 4) + weight + e * Cout * Cin, "flops": 4 * T * Cin * Cout}
    if case["op"] == "glu_down":
        return {"bytes": T * e * (2 * Cin + Cout) + weight, "flops": 2 * T * Cin * Cout + 13 * T * Cin}
    # x, dy, y and dx; the 8-bit input is kept on the way
    return {"bytes": T * Cin * e * 6 + T * (2 * Cin + 4), "flops": 30 * T * Cin}


# ------------------------------------------------------------------ 64 bits

def _quant64(x):
    """What the 8-bit form of x [C, P] (64 bits) stands for: whole multiples of the token's scale."""
    amax = torch.maximum(x.max(0).values, -x.min(0).values).clamp_min(AMAX_FLOOR)
    return (x * 127).div_(amax).round_(), amax / 127


def _glu64(x, act):
    """act(gate) value of x [2C, P], with both derivatives."""
    g, v = x.chunk(2)
    if act == "silu":
        s = torch.sigmoid(g)
        a, da = g * s, s + g * s * torch.sigmoid(-g)
    else:
        cdf = torch.special.ndtr(g)
        a, da = g * cdf, cdf + g * torch.exp(-g * g / 2) * (2 * math.pi) ** -0.5
    return a * v, v * da, a


def exact(case, seed):
    """The definition in 64 bits, sample by sample; rows are the tokens of one sample."""
    s = _inputs(case, seed)
    rows = case["P"] == 1

    def samples(t):
        return [t[:, :, 0].t()] if rows else list(t)

    def joined(parts):
        return parts[0].t()[:, :, None] if rows else torch.stack(parts)

    if case["Cout"]:
        W = s["W"].double() * s["wscale"].double()[:, None]
    if case["op"] == "linear_bwd":
        scale = s["scale"].t() if rows else s["scale"]
        dx, dW = [], torch.zeros_like(W)
        for dy, q, sc in zip(samples(s["dy"]), samples(s["q"]), scale):
            dy = dy.double()
            dx.append(W.t() @ dy)
            dW += dy @ (q.double() * sc.double()).t()
        return {"dx": joined(dx), "dW": dW}
    out = {"y": [], "dx": []}
    for i, x in enumerate(samples(s["x"])):
        x = x.double()
        if case["op"] == "glu_train":
            out["y"].append(_glu64(x, case["act"])[0])
            q, scale = _quant64(x)
            _, dg, dv = _glu64(q * scale, case["act"])
            out["dx"].append(torch.cat([dg, dv]) * samples(s["dy"])[i].double().repeat(2, 1))
            continue
        q, scale = _quant64(x if case["op"] == "linear" else _glu64(x, case["act"])[0])
        out["y"].append((W @ q) * scale)
    return {k: joined(v) for k, v in out.items() if v}
