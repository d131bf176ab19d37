"""Timing cases of the gated feed-forward block and its gradient, and of the
orthogonalised update of a weight matrix.

A case is one call of one operator.  ``run`` computes it in plain torch
operations in FP32, or, with ``own`` set, by the library's call; ``exact``
gives the same outputs in FP64 straight from the definition.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-7
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # of the orthogonalisation's polynomial a s + b s^3 + c s^5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one generated token through a small block: latency
        dict(name="ffn_token_small", op="ffn", T=1, D=1024, F=2560, type="bf16", act="silu", train=False),
        # one generated token through a full-size block: the weights' bytes
        dict(name="ffn_token", op="ffn", T=1, D=5120, F=12800, type="bf16", act="silu", train=False),
        # a batch of sequences that each generate a token
        dict(name="ffn_decode_batch", op="ffn", T=48, D=5120, F=12800, type="bf16", act="silu", train=False),
        # a ragged micro-batch with odd sizes in FP16
        dict(name="ffn_ragged", op="ffn", T=1000, D=1285, F=3427, type="fp16", act="gelu", train=True),
        # the training profile's tokens through a sublayer
        dict(name="ffn_batch", op="ffn", T=4096, D=5120, F=12800, type="bf16", act="silu", train=True),
        # the gradient of a short fine-tuning batch through a small block
        dict(name="ffn_grad_short", op="ffn_grad", T=256, D=1024, F=2560, type="bf16", act="silu", add=False),
        # the gradient of the ragged micro-batch, added to gradients held in the weights' type
        dict(name="ffn_grad_ragged", op="ffn_grad", T=1000, D=1285, F=3427, type="fp16", act="gelu", add=True),
        # the gradient of the training profile's tokens
        dict(name="ffn_grad_batch", op="ffn_grad", T=4096, D=5120, F=12800, type="bf16", act="silu", add=False),
        # the update of the projection's weight of four streams of 5120: a few long rows
        dict(name="orth_projection", op="orth", m=24, n=20480, type="fp32"),
        # odd sizes, wide
        dict(name="orth_ragged", op="orth", m=1285, n=3427, type="fp32"),
        # a square weight, its gradient as the backward writes it
        dict(name="orth_square", op="orth", m=5120, n=5120, type="bf16"),
        # the full-size block's gate projection, momentum in FP32, tall
        dict(name="orth_tall", op="orth", m=12800, n=5120, type="fp32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """Sizes over the whole range; most are multiples of 8, some of 64, some odd."""
    v, step = _log(rng, low, high), rng.choice([1, 8, 8, 64])
    return max(low, v // step * step) if step > 1 else v | 1


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "orth"])
    if op == "orth":
        m, n = _size(rng, 16, 8192), _size(rng, 16, 12800)
        if rng.random() < 0.5:
            m, n = n, m
        case = dict(op=op, m=m, n=n, type=rng.choice(["bf16", "fp16", "fp32", "fp32"]))
        while work(case)["flops"] > 5 * (3 * 12800 + 5120) * 5120 ** 2:
            case["m" if m > n else "n"] //= 2
        return case
    D, F = _size(rng, 64, 8192), _size(rng, 64, 16384)
    T = _log(rng, 1, 8192) if rng.random() < 0.7 else _log(rng, 1, 64)
    T = max(1, min(T, 4096 * 5120 * 12800 // (D * F)))
    case = dict(op=op, T=T, D=D, F=F, type=rng.choice(["bf16", "bf16", "fp16"]), act=rng.choice(["silu", "silu", "gelu"]))
    case["train" if op == "ffn" else "add"] = rng.random() < 0.5
    return case


def work(case):
    c = case
    if c["op"] == "orth":
        s, l = sorted((c["m"], c["n"]))
        # X X^T and its square are symmetric: half of their products
        return dict(bytes=s * l * (BYTES[c["type"]] + 2), flops=5 * (3 * s * s * l + s ** 3))
    T, D, F = c["T"], c["D"], c["F"]
    if c["op"] == "ffn":
        return dict(bytes=4 * T * D + 6 * D * F + (4 * T * F if c["train"] else 0), flops=6 * T * D * F)
    return dict(bytes=6 * T * D + 4 * T * F + (18 if c["add"] else 12) * D * F, flops=12 * T * D * F)


# ---------------------------------------------------------------- inputs
def _normal(shape, g, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "orth":
        # a matrix's gradient: a few strong directions of falling size, and noise in all
        m, n = c["m"], c["n"]
        r = max(1, min(m, n, 96) // 2)
        size = 0.5 * torch.arange(1, r + 1, device=DEV) ** -0.75
        G = (_normal((m, r), g) * size) @ _normal((r, n), g) + _normal((m, n), g)
        s["G"] = (1e-3 * G).to(TYPES[c["type"]])
        s["out"] = torch.empty(m, n, device=DEV, dtype=torch.bfloat16)
        return s
    T, D, F, dtype = c["T"], c["D"], c["F"], TYPES[c["type"]]
    # rows as a norm gives them, a few channels larger
    wide = torch.where(torch.rand(D, generator=g, device=DEV) < 0.005, 4.0, 1.0)
    s["x"] = (_normal((T, D), g) * wide).to(dtype)
    s["w_gate"], s["w_up"] = (_normal((F, D), g, D ** -0.5).to(dtype) for _ in range(2))
    s["w_down"] = _normal((D, F), g, F ** -0.5).to(dtype)
    if c["op"] == "ffn":
        s["y"] = torch.empty(T, D, device=DEV, dtype=dtype)
        s["gate"], s["up"] = (torch.empty(T, F, device=DEV, dtype=dtype) if c["train"] else None for _ in range(2))
        return s
    s["gate"], s["up"] = (_normal((T, F), g).to(dtype) for _ in range(2))
    s["grad_y"] = _normal((T, D), g, 1e-2).to(dtype)
    s["grad_x"] = torch.empty(T, D, device=DEV, dtype=dtype)
    for k, shape in (("w_gate", (F, D)), ("w_up", (F, D)), ("w_down", (D, F))):
        s["grad_" + k] = _normal(shape, g, 0.1).to(dtype) if c["add"] else torch.empty(shape, device=DEV, dtype=dtype)
    if c["add"]:   # what earlier micro-batches left, kept apart so that a pass can be repeated
        s["before"] = [s["grad_" + k].clone() for k in ("w_gate", "w_up", "w_down")]
    return s


# ---------------------------------------------------------------- plain form
def _act(v, kind):
    """The activation and its derivative."""
    if kind == "silu":
        q = 1.0 / (1.0 + torch.exp(-v))
        return v * q, q * (1.0 + v * (1.0 - q))
    p = 0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5))
    return v * p, p + v * torch.exp(-0.5 * v * v) * (2.0 * math.pi) ** -0.5


def _plain(s):
    c = s["case"]
    if c["op"] == "orth":
        a, b, k = COEFFICIENTS
        X = s["G"].float()
        X = X / (X.double().square().sum().sqrt().float() + EPS)
        X = X.t() if c["m"] > c["n"] else X
        for _ in range(5):
            A = X @ X.t()
            X = a * X + (b * A + k * (A @ A)) @ X
        return (X.t() if c["m"] > c["n"] else X).to(torch.bfloat16).contiguous()
    dtype = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    if c["op"] == "ffn":
        g, u = x @ wg.t(), x @ wu.t()
        y = (_act(g, c["act"])[0] * u) @ wd.t()
        return (y.to(dtype), g.to(dtype), u.to(dtype)) if c["train"] else y.to(dtype)
    g, u, dy = s["gate"].float(), s["up"].float(), s["grad_y"].float()
    f, df = _act(g, c["act"])
    da = dy @ wd
    dg, du = da * u * df, da * f
    out = [dg.t() @ x, du.t() @ x, dy.t() @ (f * u)]
    if c["add"]:
        out = [o + b.float() for o, b in zip(out, s["before"])]
    return (dg @ wg + du @ wu).to(dtype), *(o.to(dtype) for o in out)


# ---------------------------------------------------------------- the library's calls
def _workspace(s, size, *args):
    """The scratch a user's program keeps with its buffers, made at the first pass."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size(*args), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _call(s):
    import rms_backward_gb300 as m
    c = s["case"]
    if c["op"] == "orth":
        ws = _workspace(s, m.mhc_orthogonalize_workspace_bytes, c["m"], c["n"])
        m.mhc_orthogonalize(s["G"], s["out"], ws, eps=EPS)
        return s["out"]
    weights = s["w_gate"], s["w_up"], s["w_down"]
    if c["op"] == "ffn":
        ws = _workspace(s, m.mhc_ffn_forward_workspace_bytes, c["T"], c["D"], c["F"])
        m.mhc_ffn_forward(s["x"], *weights, s["y"], ws, s["gate"], s["up"], activation=c["act"])
        return (s["y"], s["gate"], s["up"]) if c["train"] else s["y"]
    ws = _workspace(s, m.mhc_ffn_backward_workspace_bytes, c["T"], c["D"], c["F"])
    grads = s["grad_w_gate"], s["grad_w_up"], s["grad_w_down"]
    if c["add"]:
        for g, b in zip(grads, s["before"]):
            g.copy_(b)
    m.mhc_ffn_backward(s["x"], *weights, s["gate"], s["up"], s["grad_y"], s["grad_x"], *grads, ws, activation=c["act"],
                       accumulate=c["add"])
    return (s["grad_x"], *grads)


def run(state):
    return _call(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    if work(c)["flops"] > 1.2e13:
        return None
    s = prepare(c, seed)
    d = lambda k: s[k].to(torch.float64)  # noqa: E731
    if c["op"] == "orth":
        # by the smaller side: X p(X^T X) or p(X X^T) X with p(t) = a + b t + c t^2
        X = d("G")
        X /= torch.linalg.vector_norm(X) + EPS
        a, b, k = COEFFICIENTS
        eye = torch.eye(min(X.shape), dtype=torch.float64, device=DEV)
        for _ in range(5):
            t = torch.einsum("ij,ik->jk", X, X) if c["m"] > c["n"] else torch.einsum("ij,kj->ik", X, X)
            p = torch.addmm(a * eye + b * t, t, t, alpha=k)
            X = X @ p if c["m"] > c["n"] else p @ X
        return X
    x, wg, wu, wd = d("x"), d("w_gate"), d("w_up"), d("w_down")
    normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device=DEV), 1.0)
    lin = torch.nn.functional.linear
    if c["op"] == "ffn":
        g, u = lin(x, wg), lin(x, wu)
        y = lin((torch.sigmoid(g) if c["act"] == "silu" else normal.cdf(g)) * g * u, wd)
        return (y, g, u) if c["train"] else y
    g, u, dy = d("gate"), d("up"), d("grad_y")
    if c["act"] == "silu":
        q = torch.sigmoid(g)
        slope = q + g * q * torch.sigmoid(-g)
    else:
        q = normal.cdf(g)
        slope = q + g * normal.log_prob(g).exp()
    da = torch.einsum("td,df->tf", dy, wd)
    dwd = torch.einsum("td,tf->df", dy, q * g * u)
    du, dg = da * q * g, da * slope * u
    del da, q, slope
    dx = dg @ wg
    dx += du @ wu
    out = [torch.einsum("tf,td->fd", v, x) for v in (dg, du)] + [dwd]
    if c["add"]:
        out = [o + b.to(torch.float64) for o, b in zip(out, s["before"])]
    return (dx, *out)
