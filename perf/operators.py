"""Measured cases of the operators around the convolution in a training step.

Channel norm (``disco_rms_norm``): the sum of a layer's output and the residual
stream, its root-mean-square norm over the channels of each pixel, and an
optional copy in 8 bits (e4m3) with a scale for each group of channels, which a
training program keeps for the backward pass in place of the 16-bit tensor.
Its gradient (``disco_rms_norm_bwd``) and the return from 8 bits
(``disco_dequant_e4m3``).  Activations are [B, C, P], P the pixels of a grid;
P = 1 is the layout of rows of features.

Gradient norm (``disco_grad_norm_clip``): the Euclidean norm over all gradients
of a model and the gradients scaled down to a largest norm, written to the
optimizer's flat buffer.

``run`` computes a pass in plain torch operations in 32 bits, or with ``own``
by the library; ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def _norm(name, B, C, P, dtype, residual=True, y=True, q=False, group=0):
    return {"name": name, "op": "norm", "B": B, "C": C, "P": P, "dtype": dtype, "residual": residual, "y": y, "q": q,
            "group": group}


def _bwd(name, B, C, P, dtype, dh=True):
    return {"name": name, "op": "norm_bwd", "B": B, "C": C, "P": P, "dtype": dtype, "dh": dh}


def _clip(name, count, Cout, Cin, K, dtype, out, ragged=False):
    return {"name": name, "op": "clip", "count": count, "Cout": Cout, "Cin": Cin, "K": K, "dtype": dtype, "out": out,
            "ragged": ragged}


def listed():
    return [
        # one pooled feature vector for each of 16 samples before a head: the latency of a call
        _norm("norm rows 16x512", 16, 512, 1, "bf16"),
        # a residual stack at the library's 512-channel shape on the 360 x 720 grid
        _norm("norm 512x360x720", 1, 512, 360 * 720, "bf16"),
        # the same step at 2 x 128 channels, with the 8-bit copy kept for the weight gradient
        _norm("norm+q8 2x128x361x720", 2, 128, 361 * 720, "bf16", q=True, group=32),
        # first norm of a stack on an odd grid (odd pixel count: no row but the first is aligned), nothing to add
        _norm("norm odd 3x80x181x361", 3, 80, 181 * 361, "f16", residual=False),
        # per-pixel features gathered into rows (a point head): only the 8-bit form is kept
        _norm("norm+q8 rows 16384x2048", 16384, 2048, 1, "bf16", y=False, q=True, group=128),
        # the stored 8-bit copy back in 16 bits, for the weight gradient
        {"name": "dequant 2x128x361x720", "op": "dequant", "B": 2, "C": 128, "P": 361 * 720, "dtype": "bf16", "group": 32},
        # gradients of the same norms: a small grid in 32 bits, the large stack, rows
        _bwd("bwd 4x32x64x128", 4, 32, 64 * 128, "f32"),
        _bwd("bwd 512x360x720", 1, 512, 360 * 720, "bf16"),
        _bwd("bwd rows 16384x2048", 16384, 2048, 1, "bf16", dh=False),
        # a small model: 8 weights of 64 channels and 3 radial filters, clipped in 32 bits
        _clip("clip 8x[64,64,3]", 8, 64, 64, 3, "f32", "f32"),
        # a large one: 16-bit weight gradients of 48 layers into the optimizer's 32-bit buffer
        _clip("clip 48x[512,512,9]", 48, 512, 512, 9, "bf16", "f32"),
        # gradients of weights, gains and biases in two types, of odd sizes
        _clip("clip 240 ragged", 240, 80, 77, 5, "mixed", "f32", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "dequant", "clip", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "clip":
        count = _log(rng, 1, 400)
        cout, cin, k = _log(rng, 4, 512), _log(rng, 3, 512), rng.randint(1, 9)
        while count * cout * cin * k > 100_000_000:
            count = (count + 1) // 2
        dtype = rng.choice(["bf16", "f16", "f32", "mixed"])
        out = "f32" if dtype == "mixed" else rng.choice(["f32", dtype])
        c = _clip("", count, cout, cin, k, dtype, out, ragged=rng.random() < 0.5)
        del c["name"]
        return c
    if rng.random() < 0.35:  # rows
        P, C, B = 1, _log(rng, 3, 16384), _log(rng, 1, 65536)
        while B * C > 60_000_000:
            B = (B + 1) // 2
    else:
        nlat = _log(rng, 4, 721)
        P = nlat * (2 * nlat if rng.random() < 0.6 else nlat + rng.randint(0, 2 * nlat))
        C, B = _log(rng, 3, 768), _log(rng, 1, 16)
        while B * C * P > 60_000_000:
            B, C = (B // 2, C) if B > 1 else (1, (C + 1) // 2)
    c = {"op": op, "B": B, "C": C, "P": P, "dtype": dtype}
    group = rng.choice([0, 16, 32, 128, rng.randint(1, max(1, C))])
    if op == "norm":
        q = rng.random() < 0.5
        c.update(residual=rng.random() < 0.7, y=not q or rng.random() < 0.6, q=q, group=group if q else 0)
    elif op == "norm_bwd":
        c.update(dh=rng.random() < 0.7)
    else:
        c.update(dtype=rng.choice(["bf16", "f16"]), group=group)
    return c


def _grad_sizes(case):
    full = case["Cout"] * case["Cin"] * case["K"]
    if not case["ragged"]:
        return [full] * case["count"]
    # weights of growing fan-in, gains and biases, as the layers of one model have them
    sizes = []
    for i in range(case["count"]):
        sizes.append((full * (i + 3) // (case["count"] + 2), case["Cout"], 2 * case["Cin"] + 1)[i % 3])
    return [max(1, n) for n in sizes]


def _grad_dtypes(case):
    if case["dtype"] != "mixed":
        return [case["dtype"]] * case["count"]
    return [("bf16", "f32", "f32")[i % 3] for i in range(case["count"])]


def _group(case):
    return case["group"] if 0 < case["group"] < case["C"] else case["C"]


def _groups(case):
    return -(-case["C"] // _group(case))


def _inputs(case, seed):
    """The tensors of a case, made on the GPU from the seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "clip":
        sizes, kinds = _grad_sizes(case), _grad_dtypes(case)
        # gradients of one model differ in size from layer to layer
        flat, level = randn(sum(sizes)), torch.rand(len(sizes), generator=g, device="cuda").mul(4).sub(6).exp()
        flat *= level.repeat_interleave(torch.tensor(sizes, device="cuda"), output_size=sum(sizes))
        return {"grads": [v.to(DTYPES[k], copy=True) for v, k in zip(flat.split(sizes), kinds)], "max_norm": 1.0}
    B, C, P, dt = case["B"], case["C"], case["P"], DTYPES[case["dtype"]]
    gain = (1 + 0.1 * randn(C)).to(dt)
    if case["op"] == "dequant":
        q = (100 * randn(B, C, P)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"q": q, "scale": 0.002 + 0.01 * torch.rand((B, _groups(case), P), generator=g, device="cuda")}
    if case["op"] == "norm":
        return {"x": randn(B, C, P).to(dt), "weight": gain, "residual": (3 * randn(B, C, P)).to(dt) if case["residual"] else None}
    # the residual stream's channels differ in size, its gradient is small
    return {"dy": (1e-2 * randn(B, C, P)).to(dt), "h": (randn(B, C, P) * (0.5 + 3 * torch.rand((C, 1), generator=g, device="cuda"))).to(dt),
            "weight": gain, "dh": (1e-2 * randn(B, C, P)).to(dt) if case["dh"] else None}


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    # what the program owns: output buffers, and for the library's calls its workspace and its plan of the gradient list
    if case["op"] == "clip":
        s["out"] = torch.empty(sum(_grad_sizes(case)), dtype=DTYPES[case["out"]], device="cuda")
        s["norm"] = torch.empty((), dtype=torch.float32, device="cuda")
        if own:
            import sparse_spherical_convolution_gb300 as d
            s["plan"] = d.GradPlan(s["grads"], list(s["out"].split(_grad_sizes(case))))
            s["workspace"] = torch.empty(d.disco_grad_workspace_bytes(s["plan"].c), dtype=torch.uint8, device="cuda")
        return s
    B, C, P, dt = case["B"], case["C"], case["P"], DTYPES[case["dtype"]]
    new = lambda d=dt: torch.empty((B, C, P), dtype=d, device="cuda")  # noqa: E731
    if case["op"] == "norm":
        s["h"] = new() if case["residual"] else None
        s["y"] = new() if case["y"] else None
        s["q"] = new(torch.float8_e4m3fn) if case["q"] else None
        s["scale"] = torch.empty((B, _groups(case), P), dtype=torch.float32, device="cuda") if case["q"] else None
    elif case["op"] == "norm_bwd":
        s["dx"], s["dweight"] = new(), torch.empty(C, dtype=dt, device="cuda")
        if own:
            import sparse_spherical_convolution_gb300 as d
            n = d.disco_rms_norm_bwd_workspace_bytes(B, C, P, d.dtype_code(dt))
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    else:
        s["x"] = new()
    return s


def run(s):
    case = s["case"]
    if own:
        return _run_library(s, case)
    if case["op"] == "clip":
        flat = torch.cat([g.float() for g in s["grads"]])
        norm = flat.square().sum().sqrt()
        coef = torch.where(norm <= s["max_norm"], torch.ones_like(norm), s["max_norm"] / norm)
        return {"norm": norm, "out": (flat * coef).to(DTYPES[case["out"]])}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "dequant":
        G = _group(case)
        return {"x": (s["q"].float() * s["scale"].repeat_interleave(G, 1)[:, :case["C"]]).to(dt)}
    w = s["weight"].float()[:, None]
    if case["op"] == "norm_bwd":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        n = h * r
        g = dy * w
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * n).sum((0, 2)).to(dt)}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
    out = {}
    if s["h"] is not None:
        out["h"] = h.to(dt)
    if s["y"] is not None:
        out["y"] = y.to(dt)
    if s["q"] is not None:
        B, C, P = y.shape
        G, n = _group(case), _groups(case)
        y = torch.nn.functional.pad(y, (0, 0, 0, n * G - C)).view(B, n, G, P)
        amax = y.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR)
        out["scale"] = (amax / E4M3_MAX).view(B, n, P)
        out["q"] = (y * (E4M3_MAX / amax)).to(torch.float8_e4m3fn).view(B, n * G, P)[:, :C].contiguous()
    return out


def _run_library(s, case):
    import sparse_spherical_convolution_gb300 as d
    if case["op"] == "clip":
        d.disco_grad_norm_clip(s["plan"].c, s["max_norm"], s["norm"], s["workspace"])
        return {"norm": s["norm"], "out": s["out"]}
    B, C, P = case["B"], case["C"], case["P"]
    if case["op"] == "dequant":
        d.disco_dequant_e4m3(s["q"], s["scale"], s["x"], B, C, P, case["group"])
        return {"x": s["x"]}
    if case["op"] == "norm_bwd":
        d.disco_rms_norm_bwd(s["dy"], s["h"], s["weight"], s["dh"], EPS, s["dx"], s["dweight"], B, C, P, s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    d.disco_rms_norm(s["x"], s["residual"], s["weight"], EPS, s["h"], s["y"], B, C, P, q=s["q"], scale=s["scale"], group=case["group"])
    return {k: s[k] for k in ("h", "y", "q", "scale") if s[k] is not None}


def work(case):
    if case["op"] == "clip":
        sizes = _grad_sizes(case)
        n = sum(sizes)
        read = sum(m * SIZES[k] for m, k in zip(sizes, _grad_dtypes(case)))
        return {"bytes": read + n * SIZES[case["out"]] + 4, "flops": 3 * n}
    B, C, P, e = case["B"], case["C"], case["P"], SIZES[case["dtype"]]
    n = B * C * P
    scales = 4 * B * P * _groups(case) if "group" in case else 0
    if case["op"] == "dequant":
        return {"bytes": n * (1 + e) + scales, "flops": n}
    if case["op"] == "norm_bwd":
        return {"bytes": n * e * (4 if case["dh"] else 3) + 2 * C * e, "flops": 10 * n}
    tensors = 1 + 2 * case["residual"] + case["y"]
    return {"bytes": n * (e * tensors + case["q"]) + C * e + (scales if case["q"] else 0), "flops": (5 + 3 * case["q"]) * n}


def _to_e4m3(v):
    """The nearest e4m3 value to each of v (64 bits, within +-448), ties to even."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(-6.0)
    step = torch.exp2(exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    """The definition in 64 bits, sample by sample."""
    s = _inputs(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        coef = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
        return {"norm": norm, "out": torch.cat([g.double().mul_(coef) for g in s["grads"]])}
    B, C, P = case["B"], case["C"], case["P"]
    G = _group(case) if "group" in case else C
    channel_group = torch.arange(C, device="cuda") // G
    parts, dweight = [], torch.zeros(C, dtype=torch.float64, device="cuda")
    step = max(1, 40_000_000 // (C * P))  # samples at a time
    for b in range(0, B, step):
        at = slice(b, b + step)
        if case["op"] == "dequant":
            parts.append({"x": s["q"][at].to(torch.float64) * s["scale"][at].double()[:, channel_group]})
            continue
        w = s["weight"].double().view(1, C, 1)
        if case["op"] == "norm_bwd":
            h, dy = s["h"][at].double(), s["dy"][at].double()
            mean = torch.einsum("bcp,bcp->bp", h, h).div_(C).add_(EPS).unsqueeze_(1)
            dot = torch.einsum("bcp,bcp->bp", dy * w, h).div_(C).unsqueeze_(1)
            dweight += torch.einsum("bcp,bcp->c", dy, h / mean.sqrt())
            dx = dy * w / mean.sqrt() - h * dot / mean ** 1.5
            parts.append({"dx": dx if s["dh"] is None else dx + s["dh"][at].double()})
            continue
        h = s["x"][at].double()
        if s["residual"] is not None:
            h += s["residual"][at].double()
        y = w * h / torch.einsum("bcp,bcp->bp", h, h).div_(C).add_(EPS).sqrt_().unsqueeze_(1)
        part = {"h": h} if case["residual"] else {}
        if case["q"]:
            amax = torch.full((y.shape[0], _groups(case), P), AMAX_FLOOR, dtype=torch.float64, device="cuda")
            amax.scatter_reduce_(1, channel_group.view(1, C, 1).expand_as(y), y.abs(), "amax")
            part["scale"] = amax / E4M3_MAX
            part["q"] = _to_e4m3(y * E4M3_MAX / amax[:, channel_group])
        if case["y"]:
            part["y"] = y
        parts.append(part)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "norm_bwd":
        out["dweight"] = dweight
    return out
