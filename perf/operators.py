"""Timing cases of the operators around the projection stage: the embedding
lookup into the residual streams, layer norm, counter-based dropout, the
stream collapse with its norm, and the stream update, with their gradients.

A case is one call of one operator.  ``run`` computes it in plain torch
operations in FP32, or, with ``own`` set, by the library's call; ``exact``
gives the same outputs in FP64 straight from the definition.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
STREAMS = 4          # residual streams; h holds 4 + 4 + 16 gates per token
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a training batch enters the streams: 16,384 tokens of hidden size 5120
        dict(name="embed_batch", op="embed", T=16384, D=5120, V=65536, n=4, type="bf16", wide=True, pad=0.0, scale=1.0),
        # the gradient of one rank's 4,096 tokens, written over the whole table
        dict(name="embed_grad", op="embed_grad", T=4096, D=5120, V=32768, n=4, wide=True, pad=0.0, scale=1.0, add=False),
        # a ragged micro-batch with padding, added to an FP32 gradient buffer; odd hidden size, one stream
        dict(name="embed_grad_ragged", op="embed_grad", T=1000, D=1285, V=5003, n=1, wide=False, pad=0.05, scale=0.5, add=True),
        # one generated token through a norm: latency
        dict(name="norm_token", op="norm", T=1, D=5120, type="bf16"),
        # a ragged batch's norm gradient in FP32, odd hidden size
        dict(name="norm_grad_ragged", op="norm_grad", T=1000, D=1285, type="fp32"),
        # the norm's gradient at the long sublayer's 16,384 tokens
        dict(name="norm_grad_long", op="norm_grad", T=16384, D=5120, type="bf16"),
        # dropout of one sublayer's output
        dict(name="dropout_batch", op="dropout", T=4096, D=5120, type="bf16", p=0.1),
        # an odd number of FP32 activations
        dict(name="dropout_ragged", op="dropout", T=333, D=1285, type="fp32", p=0.25),
        # streams to a sublayer's normalised input, the training profile's tokens
        dict(name="collapse_batch", op="collapse", T=4096, D=5120),
        # its gradient, with the residual path's, at the long sublayer
        dict(name="collapse_grad_long", op="collapse_grad", T=16384, D=5120),
        # one generated token's stream update, no dropout: latency
        dict(name="update_token", op="update", T=1, D=5120, p=0.0),
        # the update's gradient, the training profile's tokens
        dict(name="update_grad_batch", op="update_grad", T=4096, D=5120, p=0.1),
    ]


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "dropout", "collapse", "collapse_grad",
                     "update", "update_grad"])
    D = int(round(math.exp(rng.uniform(math.log(64), math.log(8192)))))
    if rng.random() < 0.7:                    # most hidden sizes are multiples of 8
        g = rng.choice([8, 40, 320])
        D = max(g, D // g * g)
    T = int(round(math.exp(rng.uniform(0.0, math.log(16384)))))
    if T * D > 16384 * 5120:
        T = 16384 * 5120 // D
    case = dict(op=op, T=T, D=D)
    if op in ("embed", "embed_grad"):
        case["V"] = int(round(math.exp(rng.uniform(math.log(256), math.log(32768 if D > 2560 else 65536)))))
        case["n"] = rng.choice([1, STREAMS, STREAMS])
        case["wide"] = rng.random() < 0.7
        case["pad"] = rng.choice([0.0, 0.0, 0.1])
        case["scale"] = rng.choice([1.0, 0.5, round(math.sqrt(D), 3)])
        if op == "embed":
            case["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        else:
            case["add"] = rng.random() < 0.5
    elif op in ("norm", "norm_grad", "dropout"):
        case["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("dropout", "update", "update_grad"):
        case["p"] = rng.choice([0.0, 0.1, 0.25, 0.5]) if op != "dropout" else rng.choice([0.1, 0.25, 0.5])
    return case


def _token_weights(V):
    """Token frequencies fall off as 1 / (rank + 2.7), as words of a text do."""
    w = 1.0 / (np.arange(V) + 2.7)
    return w / w.sum()


def _distinct(c):
    """Expected number of different tokens among T (1 - pad) draws."""
    n = c["T"] * (1.0 - c["pad"])
    return max(1.0, float(-np.expm1(n * np.log1p(-_token_weights(c["V"]))).sum()))


def work(case):
    c = case
    T, D, op = c["T"], c["D"], c["op"]
    e = BYTES[c.get("type", "bf16")]
    gates = T * 24 * 4
    if op == "embed":
        idb = T * (8 if c["wide"] else 4)
        return dict(bytes=idb + _distinct(c) * D * e + 2 * T * c["n"] * D, flops=T * D)
    if op == "embed_grad":
        idb = T * (8 if c["wide"] else 4)
        table = _distinct(c) * D * 8 if c["add"] else c["V"] * D * 4
        return dict(bytes=idb + 2 * T * c["n"] * D + table, flops=T * D * (c["n"] + 1))
    if op == "norm":
        return dict(bytes=2 * T * D * e + 8 * D + 8 * T, flops=8 * T * D)
    if op == "norm_grad":
        return dict(bytes=3 * T * D * e + 12 * D + 8 * T, flops=14 * T * D)
    if op == "dropout":
        return dict(bytes=2 * T * D * e, flops=2 * T * D)
    if op == "collapse":
        return dict(bytes=10 * T * D + gates // 6 + 8 * D + 8 * T, flops=15 * T * D)
    if op == "collapse_grad":
        return dict(bytes=26 * T * D + gates + gates // 6 + 12 * D + 8 * T, flops=70 * T * D)
    if op == "update":
        return dict(bytes=18 * T * D + gates, flops=41 * T * D)
    return dict(bytes=20 * T * D + 2 * gates, flops=50 * T * D)


# ---------------------------------------------------------------- inputs
def _gates(T, g):
    """Gates as the gate step writes them: sigmoid, 2 sigmoid, and a 4 x 4
    matrix whose rows and columns have been normalised in turn 20 times."""
    l = torch.randn(T, 24, generator=g, device=DEV)
    m = torch.exp(l[:, 8:].reshape(T, 4, 4))
    for _ in range(20):
        m = m / m.sum(2, keepdim=True)
        m = m / m.sum(1, keepdim=True)
    return torch.cat([torch.sigmoid(l[:, :4]), 2 * torch.sigmoid(l[:, 4:8]), m.reshape(T, 16)], 1).contiguous()


def _activations(shape, dtype, g, scale=1.0):
    """Rows of differing size, a few channels far larger than the others."""
    T, D = shape
    x = torch.randn(T, D, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    x *= torch.where(torch.rand(D, generator=g, device=DEV) < 0.005, 8.0, 1.0)
    x += 0.1 * torch.randn(D, generator=g, device=DEV)
    return (scale * x).to(dtype)


def _mix(x, h):
    """sum_s h[:, s] x_s over the streams of x [T, 4 D], FP32."""
    T, D = x.shape[0], x.shape[1] // STREAMS
    return (x.view(T, STREAMS, D).float() * h[:, :4, None]).sum(1)


def _moments(u):
    mean = u.mean(1)
    rstd = 1.0 / torch.sqrt(((u - mean[:, None]) ** 2).mean(1) + EPS)
    return mean, rstd


def prepare(case, seed):
    c = case
    T, D, op = c["T"], c["D"], c["op"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=c)
    if op in ("embed", "embed_grad"):
        V = c["V"]
        cum = torch.from_numpy(np.cumsum(_token_weights(V))).to(DEV)
        ids = torch.searchsorted(cum, torch.rand(T, generator=g, device=DEV, dtype=torch.float64)).clamp_(max=V - 1)
        if c["pad"]:
            ids = torch.where(torch.rand(T, generator=g, device=DEV) < c["pad"], -1, ids)
        s["ids"] = ids.to(torch.int64 if c["wide"] else torch.int32)
        if op == "embed":
            s["table"] = torch.empty(V, D, device=DEV, dtype=TYPES[c["type"]]).normal_(0.0, 0.02, generator=g)
            s["x"] = torch.empty(T, c["n"] * D, device=DEV, dtype=torch.bfloat16)
        else:
            s["grad_x"] = _activations((T, c["n"] * D), torch.bfloat16, g, 1e-2)
            s["grad_table"] = torch.empty(V, D, device=DEV)
            if c["add"]:
                s["grad_table"].normal_(0.0, 1e-2, generator=g)
        return s
    dtype = TYPES[c.get("type", "bf16")]
    if op in ("norm", "norm_grad", "collapse", "collapse_grad"):
        s["gamma"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
        s["beta"] = 0.1 * torch.randn(D, generator=g, device=DEV)
    if op in ("dropout", "update", "update_grad"):
        s["rng"] = torch.randint(-2**62, 2**62, (2,), generator=g, device=DEV, dtype=torch.int64)
    if op in ("norm", "norm_grad", "dropout"):
        s["x"] = _activations((T, D), dtype, g)
        s["y"] = torch.empty_like(s["x"])
    else:
        s["x"] = _activations((T, STREAMS * D), dtype, g)
        s["h"] = _gates(T, g)
    if op in ("norm", "collapse"):
        s["mean"], s["rstd"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        s["y"] = torch.empty(T, D, device=DEV, dtype=dtype)
    if op in ("norm_grad", "collapse_grad"):
        s["mean"], s["rstd"] = _moments(s["x"].float() if op == "norm_grad" else _mix(s["x"], s["h"]))
        s["grad_y"] = _activations((T, D), dtype, g, 1e-2)
        s["grad_x"] = torch.empty_like(s["x"])
        s["grad_gamma"], s["grad_beta"] = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    if op in ("collapse_grad", "update_grad"):
        s["grad_x_out"] = _activations((T, STREAMS * D), dtype, g, 1e-2)
        s["grad_h"] = torch.zeros(T, 24, device=DEV)
    if op in ("update", "update_grad"):
        s["y"] = _activations((T, D), dtype, g)
    if op == "update":
        s["x_out"] = torch.empty_like(s["x"])
    if op == "update_grad":
        s["grad_y"] = torch.empty_like(s["y"])
    return s


# ---------------------------------------------------------------- plain form
MASK32 = 0xFFFFFFFF


def _round(c0, c1, c2, c3, k0, k1):
    """One round of Philox4x32 on 32-bit words held in int64 (products wrap at 64 bits)."""
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return ((b >> 32) & MASK32) ^ c1 ^ k0, b & MASK32, ((a >> 32) & MASK32) ^ c3 ^ k1, a & MASK32


def _random_words(count, rng, sequence=0):
    """`count` 32-bit words of Philox4x32-10: counter (i // 4, rng[1] + sequence), key rng[0]."""
    i = torch.arange(-(-count // 4), device=DEV, dtype=torch.int64)
    q = rng[1] + sequence
    c = (i & MASK32, i >> 32, (q & MASK32).expand_as(i), ((q >> 32) & MASK32).expand_as(i))
    k0, k1 = rng[0] & MASK32, (rng[0] >> 32) & MASK32
    for r in range(10):
        c = _round(*c, (k0 + r * 0x9E3779B9) & MASK32, (k1 + r * 0xBB67AE85) & MASK32)
    return torch.stack(c, 1).reshape(-1)[:count]


def _kept(shape, p, rng):
    """Where an element is kept, and what it is multiplied by."""
    p = np.float32(p)
    words = _random_words(shape[0] * shape[1], rng).view(shape)
    return words >= int(np.floor(np.float64(p) * 2.0**32 + 0.5)), float(np.float32(1) / (np.float32(1) - p))


def _drop(v, p, rng):
    if p == 0:
        return v
    keep, scale = _kept(v.shape, p, rng)
    return torch.where(keep, v * scale, 0.0)


def _norm_grad(u, gy, s):
    """Gradients of the norm's input (FP32), gamma and beta."""
    xhat = (u - s["mean"][:, None]) * s["rstd"][:, None]
    gh = gy * s["gamma"]
    du = s["rstd"][:, None] * (gh - gh.mean(1, keepdim=True) - xhat * (gh * xhat).mean(1, keepdim=True))
    return du, (gy * xhat).sum(0), gy.sum(0)


def _plain(s):
    c = s["case"]
    T, D, op = c["T"], c["D"], c["op"]
    if op == "embed":
        ok = (s["ids"] >= 0) & (s["ids"] < c["V"])
        rows = s["table"][torch.where(ok, s["ids"], 0)].float() * c["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(torch.bfloat16).repeat(1, c["n"])
    if op == "embed_grad":
        ok = (s["ids"] >= 0) & (s["ids"] < c["V"])
        rows = s["grad_x"].view(T, c["n"], D).float().sum(1) * c["scale"]
        if not c["add"]:
            s["grad_table"].zero_()
        return s["grad_table"].index_add_(0, torch.where(ok, s["ids"], 0), torch.where(ok[:, None], rows, 0.0))
    if op == "norm" or op == "collapse":
        u = s["x"].float() if op == "norm" else _mix(s["x"], s["h"])
        mean, rstd = _moments(u)
        y = (u - mean[:, None]) * rstd[:, None] * s["gamma"] + s["beta"]
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_grad":
        du, gg, gb = _norm_grad(s["x"].float(), s["grad_y"].float(), s)
        return du.to(s["x"].dtype), gg, gb
    if op == "dropout":
        return _drop(s["x"].float(), c["p"], s["rng"]).to(s["x"].dtype)
    h = s["h"]
    if op == "collapse_grad":
        x = s["x"].view(T, STREAMS, D).float()
        du, gg, gb = _norm_grad(_mix(s["x"], h), s["grad_y"].float(), s)
        back = torch.bmm(h[:, 8:].reshape(T, 4, 4).transpose(1, 2), s["grad_x_out"].view(T, STREAMS, D).float())
        gx = (back + h[:, :4, None] * du[:, None, :]).to(torch.bfloat16).view(T, STREAMS * D)
        gh = torch.cat([(x * du[:, None, :]).sum(2), torch.zeros(T, 20, device=DEV)], 1)
        return gx, gh, gg, gb
    y = _drop(s["y"].float(), c["p"], s["rng"])
    if op == "update":
        out = torch.bmm(h[:, 8:].reshape(T, 4, 4), s["x"].view(T, STREAMS, D).float())
        return (out + h[:, 4:8, None] * y[:, None, :]).to(torch.bfloat16).view(T, STREAMS * D)
    go = s["grad_x_out"].view(T, STREAMS, D).float()
    gy = _drop((go * h[:, 4:8, None]).sum(1), c["p"], s["rng"]).to(torch.bfloat16)
    ghp = (go * y[:, None, :]).sum(2)
    ghr = torch.bmm(go, s["x"].view(T, STREAMS, D).float().transpose(1, 2)).reshape(T, 16)
    return gy, torch.cat([torch.zeros(T, 4, device=DEV), ghp, ghr], 1)


# ---------------------------------------------------------------- the library's calls
def _workspace(s, size, *args):
    """The scratch a user's program keeps with its buffers, made at the first pass."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size(*args), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _call(s):
    import rms_backward_gb300 as m
    c = s["case"]
    op = c["op"]
    if op == "embed":
        m.mhc_embed_forward(s["ids"], s["table"], s["x"], scale=c["scale"])
        return s["x"]
    if op == "embed_grad":
        ws = _workspace(s, m.mhc_embed_workspace_bytes, c["T"], c["V"], c["D"])
        m.mhc_embed_backward(s["ids"], s["grad_x"], s["grad_table"], ws, scale=c["scale"], accumulate=c["add"])
        return s["grad_table"]
    if op == "norm":
        m.mhc_layernorm_forward(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if op == "norm_grad":
        ws = _workspace(s, m.mhc_layernorm_workspace_bytes, c["T"], c["D"])
        m.mhc_layernorm_backward(s["x"], s["grad_y"], s["gamma"], s["mean"], s["rstd"], s["grad_x"],
                                 s["grad_gamma"], s["grad_beta"], ws)
        return s["grad_x"], s["grad_gamma"], s["grad_beta"]
    if op == "dropout":
        m.mhc_dropout(s["x"], s["y"], s["rng"], p=c["p"])
        return s["y"]
    if op == "collapse":
        m.mhc_collapse_norm_forward(s["x"], s["h"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if op == "collapse_grad":
        ws = _workspace(s, m.mhc_collapse_norm_workspace_bytes, c["T"], c["D"])
        m.mhc_collapse_norm_backward(s["x"], s["h"], s["grad_y"], s["gamma"], s["mean"], s["rstd"], s["grad_x"],
                                     s["grad_h"], s["grad_gamma"], s["grad_beta"], ws, grad_x_out=s["grad_x_out"])
        return s["grad_x"], s["grad_h"], s["grad_gamma"], s["grad_beta"]
    if op == "update":
        m.mhc_update_forward(s["x"], s["y"], s["h"], s["x_out"], s["rng"], p=c["p"])
        return s["x_out"]
    m.mhc_update_backward(s["x"], s["y"], s["h"], s["grad_x_out"], s["grad_y"], s["grad_h"], s["rng"], p=c["p"])
    return s["grad_y"], s["grad_h"]


def run(state):
    return _call(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def _philox_u64(count, rng):
    """The same words with unsigned 64-bit integers on the host (numpy), from
    the generator's definition: each round multiplies words 0 and 2 by the two
    constants and adds the two Weyl constants to the key."""
    key, step = (int(v) % 2**64 for v in rng.tolist())
    i = np.arange(-(-count // 4), dtype=np.uint64)
    lo = np.uint64(MASK32)
    ctr = [i & lo, i >> np.uint64(32), np.full_like(i, step & MASK32), np.full_like(i, step >> 32)]
    k = [key & MASK32, key >> 32]
    for _ in range(10):
        m0, m1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(m1 >> np.uint64(32)) ^ ctr[1] ^ np.uint64(k[0]), m1 & lo,
               (m0 >> np.uint64(32)) ^ ctr[3] ^ np.uint64(k[1]), m0 & lo]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    return np.stack(ctr, 1).reshape(-1)[:count]


def _factor(shape, p, rng):
    """What each element is multiplied by: 0 or 1 / (1 - p), in FP64."""
    p = float(np.float32(p))
    if p == 0:
        return torch.ones(shape, dtype=torch.float64, device=DEV)
    dropped = _philox_u64(shape[0] * shape[1], rng) < np.uint64(math.floor(p * 2.0**32 + 0.5))
    return torch.from_numpy(np.where(dropped, 0.0, 1.0 / (1.0 - p))).to(DEV).view(shape)


def exact(case, seed):
    c = case
    T, D, op = c["T"], c["D"], c["op"]
    s = prepare(c, seed)
    f = lambda k: s[k].to(torch.float64)  # noqa: E731
    if op == "embed":
        t = torch.cat([f("table"), torch.zeros(1, D, dtype=torch.float64, device=DEV)])   # row V: no token
        ids = s["ids"].long()
        rows = t[torch.where((ids < 0) | (ids >= c["V"]), c["V"], ids)] * c["scale"]
        return torch.cat([rows] * c["n"], 1)
    if op == "embed_grad":
        ids = s["ids"].long()
        out = torch.zeros(c["V"] + 1, D, dtype=torch.float64, device=DEV)                 # row V: no token
        ids = torch.where((ids < 0) | (ids >= c["V"]), c["V"], ids)
        for k in range(c["n"]):
            out.index_add_(0, ids, f("grad_x")[:, k * D:(k + 1) * D] * c["scale"])
        return out[:c["V"]] + (f("grad_table") if c["add"] else 0.0)
    if op == "dropout":
        return f("x") * _factor((T, D), c["p"], s["rng"])
    x, h = f("x"), f("h") if "h" in s else None
    if op in ("norm", "collapse", "norm_grad", "collapse_grad"):
        u = x
        if h is not None:
            u = sum(h[:, k:k + 1] * x[:, k * D:(k + 1) * D] for k in range(4))
        if op in ("norm", "collapse"):
            var, mean = torch.var_mean(u, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            return torch.addcmul(f("beta"), f("gamma"), (u - mean[:, None]) * rstd[:, None]), mean, rstd
        mean, rstd, gy = f("mean")[:, None], f("rstd")[:, None], f("grad_y")
        z = (u - mean) * rstd
        w = gy * f("gamma")
        du = (w - w.sum(1, keepdim=True) / D - z * ((w * z).sum(1, keepdim=True) / D)) * rstd
        gg, gb = torch.einsum("td,td->d", gy, z), gy.sum(0)
        if op == "norm_grad":
            return du, gg, gb
        del z, w, u
        gx = torch.empty_like(x)
        gh = torch.zeros(T, 24, dtype=torch.float64, device=DEV)
        go = f("grad_x_out")
        for j in range(4):
            cols = slice(j * D, (j + 1) * D)
            gx[:, cols] = h[:, j:j + 1] * du
            for i in range(4):
                gx[:, cols] += h[:, 8 + 4 * i + j, None] * go[:, i * D:(i + 1) * D]
            gh[:, j] = (x[:, cols] * du).sum(1)
        return gx, gh, gg, gb
    m = _factor((T, D), c["p"], s["rng"])
    y = f("y") * m
    if op == "update":
        return torch.cat([sum(h[:, 8 + 4 * i + j, None] * x[:, j * D:(j + 1) * D] for j in range(4))
                          + h[:, 4 + i, None] * y for i in range(4)], 1)
    go = f("grad_x_out")
    gy = m * sum(h[:, 4 + i, None] * go[:, i * D:(i + 1) * D] for i in range(4))
    gh = torch.zeros(T, 24, dtype=torch.float64, device=DEV)
    for i in range(4):
        gi = go[:, i * D:(i + 1) * D]
        gh[:, 4 + i] = (gi * y).sum(1)
        for j in range(4):
            gh[:, 8 + 4 * i + j] = (gi * x[:, j * D:(j + 1) * D]).sum(1)
    return gy, gh
