"""Norms and dropout between message layers: the measured cases and their plain forms.

Operators (the framework's entry points of the same names):
  layer_norm           s = residual + dropout(x), y = (s - mean) / sqrt(var + eps) * w + b over each row [rows, cols]
  layer_norm_backward  its gradients: of the sum, of x behind the dropout, of w and b
  degree_norm          the rotation-equivariant form on node features [N, C, (l_max+1)^2]: degree 0 as a layer norm over
                       the channels, each degree l > 0 divided by its root mean square over channels and orders
  degree_norm_backward its gradients
  dropout              the mask from a counter-based generator (Philox4x32-10), by element or by whole channel; its
                       backward pass is the same call on the gradient

The dropout draw of unit u = column // group in row r: word (u % 8) // 2 of the Philox block with counter
(u // 8, r, offset low, offset high) and key seed; its low 16 bits for even u, its high 16 for odd u.  A unit is kept
where the draw is at least t = floor(65536 p + 1/2), and scaled by 65536 / (65536 - t).
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the scalars of a 64-atom molecule, one call of a small inference loop: latency
        dict(name="ln_f32_64x64", op="layer_norm", dtype="f32", rows=64, cols=64, pad=0, residual=False, p=0.0, group=1),
        # the hidden layer of a radial network over the edges of a 100,000-atom system
        dict(name="ln_bf16_1909372x64", op="layer_norm", dtype="bf16", rows=1909372, cols=64, pad=0, residual=False,
             p=0.0, group=1),
        # an odd width, cut out of a wider matrix (a projection that makes several things at once)
        dict(name="ln_f32_16516x131", op="layer_norm", dtype="f32", rows=16516, cols=131, pad=58, residual=False, p=0.0,
             group=1),
        # residual stream and elementwise dropout of a node update in training
        dict(name="ln_res_bf16_10000x1024", op="layer_norm", dtype="bf16", rows=10000, cols=1024, pad=0, residual=True,
             p=0.1, group=1),
        # its gradients on the edges of the dense 10,000-atom system
        dict(name="ln_bwd_bf16_477664x128", op="layer_norm_backward", dtype="bf16", rows=477664, cols=128, pad=0,
             residual=False, p=0.0, group=1),
        # an odd width with everything on: gradient from the residual stream, dropout behind
        dict(name="ln_bwd_res_f32_16516x509", op="layer_norm_backward", dtype="f32", rows=16516, cols=509, pad=0,
             residual=True, p=0.2, group=1),
        # node features of the 1000-atom layer, inference
        dict(name="deg_f32_1000x32_l3", op="degree_norm", dtype="f32", rows=1000, channels=32, l_max=3, residual=False,
             p=0.0),
        # node update of the 100,000-atom layer in training: residual stream, whole channels dropped
        dict(name="deg_res_f32_100000x64_l3", op="degree_norm", dtype="f32", rows=100000, channels=64, l_max=3,
             residual=True, p=0.1),
        # its gradients on the dense 10,000-atom layer, mixed precision
        dict(name="deg_bwd_res_bf16_10000x128_l3", op="degree_norm_backward", dtype="bf16", rows=10000, channels=128,
             l_max=3, residual=True, p=0.1),
        # gradients at degree 6, where a channel is 49 values
        dict(name="deg_bwd_f32_20000x32_l6", op="degree_norm_backward", dtype="f32", rows=20000, channels=32, l_max=6,
             residual=False, p=0.0),
        # elementwise dropout of the radial network's hidden layer, 100,000 atoms
        dict(name="drop_bf16_1909372x64", op="dropout", dtype="bf16", rows=1909372, cols=64, group=1, p=0.1),
        # whole channels of the 1000-atom layer's messages
        dict(name="drop_f32_1000x512_g16", op="dropout", dtype="f32", rows=1000, cols=512, group=16, p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "degree_norm", "degree_norm_backward", "dropout"])
    c = dict(op=op, dtype=rng.choice(["f32", "bf16"]))
    p = rng.choice([0.0, 0.05, 0.1, 0.3, 0.5])
    if op.startswith("degree"):
        c["l_max"] = rng.choice([3, 3, 4, 5, 6])
        c["channels"] = _log(rng, 4, 256)
        width = c["channels"] * (c["l_max"] + 1) ** 2
        c["rows"] = _log(rng, 1, min(100000, 30_000_000 // width))
        c["residual"], c["p"] = rng.random() < 0.5, p
        return c
    c["group"] = rng.choice([1, 1, 1, 16, 25, 49])
    c["cols"] = _log(rng, max(8, c["group"]), 8192)
    c["cols"] = max(2 if c["group"] > 1 else 8, c["cols"] // c["group"]) * c["group"]
    c["rows"] = _log(rng, 1, min(2_000_000, 30_000_000 // c["cols"]))
    c["p"] = p
    if op == "dropout":
        c["p"] = p or 0.2
        return c
    c["residual"] = rng.random() < 0.5
    c["pad"] = rng.choice([0, 0, 0, 8, 5])
    return c


# ------------------------------------------------------------------ inputs
def _width(c):
    return c["channels"] * (c["l_max"] + 1) ** 2 if "channels" in c else c["cols"]


def _rows_of(case, gen, scale=1.0):
    """[rows, width] in a matrix that is `pad` wider: a mean and a spread of each row's own; every 64th row all zero, as
    the messages into a node without neighbours are."""
    n, d, pad = case["rows"], _width(case), case.get("pad", 0)
    t = torch.randn((n, d + pad), generator=gen, device="cuda")
    if "channels" not in case and case["op"] != "dropout":
        t += 0.5 * torch.randn((n, 1), generator=gen, device="cuda")
    t *= scale * torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda"))
    t[63::64] = 0
    return t.to(TYPES[case["dtype"]])[:, :d]


def _like_features(t, case):
    return t.reshape(case["rows"], case["channels"], -1) if "channels" in case else t


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, d, dt = case["rows"], _width(case), TYPES[case["dtype"]]
    st = dict(case=dict(case), seed=(seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 64, offset=seed % 1000 + 2 ** 33)
    backward = case["op"].endswith("backward")
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    st["x"] = _like_features(_rows_of(case, gen), case)
    if case["op"].startswith("layer"):
        st["w"], st["b"] = 1 + 0.2 * rand(d), 0.1 * rand(d)
    if case["op"].startswith("degree"):
        st["w"], st["b"] = 1 + 0.2 * rand(case["l_max"] + 1, case["channels"]), 0.1 * rand(case["channels"])
    if case.get("residual"):
        st["r"] = _like_features(_rows_of(dict(case, pad=0), gen), case)  # the residual stream, or its gradient
    if backward:
        st["g"] = _like_features(_rows_of(dict(case, pad=0), gen, 0.1), case)
        st["stats"] = _stats(st["x"].double(), case).float()
    # the buffers that a training or inference loop keeps for the results
    like = lambda: torch.empty((n, d), dtype=dt, device="cuda").reshape(st["x"].shape)  # noqa: E731
    if case["op"] == "dropout":
        st["out"] = like()
    elif backward:
        st["need"] = ("x", "w", "b", "r") if _apart(case) else ("x", "w", "b")
        st["out"] = {k: like() if k in "xr" else torch.empty_like(st[k]) for k in st["need"]}
    else:
        st["need"] = ("y", "stats", "s") if _sums(case) else ("y", "stats")
        st["out"] = {k: torch.empty((n, _stats_width(case)), device="cuda") if k == "stats" else like() for k in st["need"]}
    return st


def _sums(case):
    """Whether the normalised sum is something other than x, which the backward pass then has to be given."""
    return bool(case["residual"] or case["p"])


def _apart(case):
    """Whether the gradient of the residual stream is another one than that of x."""
    return bool(case["residual"] and case["p"])


def _stats_width(case):
    return case["l_max"] + 2 if "channels" in case else 2


# ------------------------------------------------------------------ plain forms
def _philox_round(c, i, k0, k1):
    """One round on int64 words; products wrap at 64 bits, so that the high word is the product shifted down."""
    m = 0xFFFFFFFF
    a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return (((b >> 32) & m) ^ c[1] ^ ((k0 + i * 0x9E3779B9) & m), b & m,
            ((a >> 32) & m) ^ c[3] ^ ((k1 + i * 0xBB67AE85) & m), a & m)


def _keep(rows, cols, group, p, seed, offset):
    """[rows, cols] truth values: which elements the dropout keeps."""
    units = cols // group
    blocks = (units + 7) // 8
    c0 = torch.arange(blocks, device="cuda").expand(rows, blocks)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, blocks)
    m = 0xFFFFFFFF
    start = (c0, c1, torch.full_like(c0, offset & m), torch.full_like(c0, offset >> 32))
    words = functools.reduce(lambda c, i: _philox_round(c, i, seed & m, seed >> 32), range(10), start)
    words = torch.stack(words, -1)
    draws = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(rows, 8 * blocks)[:, :units]
    return (draws >= math.floor(65536 * p + 0.5)).repeat_interleave(group, 1)


def _dropped(x, st):
    """x in 32 bits with the case's dropout applied."""
    case = st["case"]
    if not case["p"]:
        return x
    k = (case["l_max"] + 1) ** 2 if "channels" in case else case["group"]
    keep = _keep(case["rows"], _width(case), k, case["p"], st["seed"], st["offset"]).reshape(x.shape)
    t = math.floor(65536 * case["p"] + 0.5)
    return torch.where(keep, x * (65536 / (65536 - t)), 0.0)


def _degrees(l_max):
    return torch.arange((l_max + 1) ** 2, device="cuda").double().sqrt().floor().long()


def _by_degree(v, l_max):
    """[N, C, K] -> [N, l_max+1]: the mean over the channels and orders of each degree."""
    which = torch.nn.functional.one_hot(_degrees(l_max)).to(v.dtype)
    return (v.mean(1)[:, :, None] * (which / which.sum(0))).sum(1)


def _stats(s, case):
    """The mean (of degree 0) and the reciprocal deviation (of each degree), [rows, 2] or [rows, l_max + 2]."""
    if "channels" not in case:
        mu = s.mean(1, keepdim=True)
        return torch.cat((mu, 1 / torch.sqrt((s - mu).square().mean(1, keepdim=True) + EPS)), 1)
    first = (torch.arange(s.shape[2], device=s.device) == 0).to(s.dtype)
    mu = s[:, :, 0].mean(1)
    v = _by_degree((s - mu[:, None, None] * first).square(), case["l_max"])
    return torch.cat((mu[:, None], 1 / torch.sqrt(v + EPS)), 1)


def _normed(s, stats, case):
    """s with its mean taken off and its deviation divided out."""
    if "channels" not in case:
        return (s - stats[:, :1]) * stats[:, 1:]
    first = (torch.arange(s.shape[2], device=s.device) == 0).to(s.dtype)
    return (s - stats[:, :1, None] * first) * stats[:, 1:][:, _degrees(case["l_max"])][:, None, :]


def _plain_forward(st):
    case, dt = st["case"], st["x"].dtype
    s = _dropped(st["x"].float(), st)
    if case["residual"]:
        s = s + st["r"].float()
    stats = _stats(s, case)
    h = _normed(s, stats, case)
    if "channels" in case:
        y = h * st["w"][_degrees(case["l_max"])].t()
        y[:, :, 0] += st["b"]
    else:
        y = h * st["w"] + st["b"]
    got = dict(y=y.to(dt), stats=stats)
    if _sums(case):
        got["s"] = s.to(dt)
    return got


def _plain_backward(st):
    case, dt, g, stats = st["case"], st["x"].dtype, st["g"].float(), st["stats"]
    h = _normed(st["x"].float(), stats, case)
    if "channels" in case:
        deg = _degrees(case["l_max"])
        first = (torch.arange(h.shape[2], device=h.device) == 0).to(h.dtype)
        a = g * st["w"][deg].t()
        mean_a = a[:, :, 0].mean(1)[:, None, None] * first
        mean_ah = _by_degree(a * h, case["l_max"])[:, deg][:, None, :]
        r = (a - mean_a - h * mean_ah) * stats[:, 1:][:, deg][:, None, :]
        dw = torch.zeros_like(st["w"]).index_add_(0, deg, (g * h).sum(0).t())
        db = g[:, :, 0].sum(0)
    else:
        a = g * st["w"]
        r = (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True)) * stats[:, 1:]
        dw, db = (g * h).sum(0), g.sum(0)
    if case["residual"]:
        r = r + st["r"].float()
    got = dict(x=_dropped(r, st).to(dt), w=dw, b=db)
    if _apart(case):
        got["r"] = r.to(dt)
    return got


def run(st):
    op = st["case"]["op"]
    if own:
        import equivariant_gnn_message_gb300 as eq

        case, group = st["case"], (st["x"].shape[2] if "channels" in st["case"] else st["case"]["group"])
        drop = eq.Dropout(p=case["p"], seed=st["seed"], offset=st["offset"], group=group) if case["p"] else None
        if op == "dropout":
            return eq.eqmp_dropout(st["x"], drop, out=st["out"])
        if op.endswith("backward"):
            call = eq.eqmp_degree_norm_backward if op == "degree_norm_backward" else eq.eqmp_layer_norm_backward
            return call(st["g"], st["x"], st["stats"], st["w"], grad_s=st.get("r"), drop=drop, need=st["need"], out=st["out"])
        call = eq.eqmp_degree_norm if op == "degree_norm" else eq.eqmp_layer_norm
        return call(st["x"], st["w"], st["b"], eps=EPS, residual=st.get("r"), drop=drop, need=st["need"], out=st["out"])
    if op == "dropout":
        return _dropped(st["x"].float(), st).to(st["x"].dtype)
    return _plain_backward(st) if op.endswith("backward") else _plain_forward(st)


# ------------------------------------------------------------------ in 64 bits
def _exact_factor(case, seed, offset):
    """[rows, width] in 64 bits: what the dropout multiplies each element by (numpy, the generator's rounds written out)."""
    rows, width = case["rows"], _width(case)
    group = (case["l_max"] + 1) ** 2 if "channels" in case else case["group"]
    units = width // group
    nb = -(-units // 8)
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    x0 = np.tile(np.arange(nb, dtype=np.uint64), rows)
    x1 = np.repeat(np.arange(rows, dtype=np.uint64), nb)
    x2 = np.full(rows * nb, offset % 2 ** 32, dtype=np.uint64)
    x3 = np.full(rows * nb, offset // 2 ** 32, dtype=np.uint64)
    ka, kb = seed % 2 ** 32, seed // 2 ** 32
    for _ in range(10):
        p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (p1 >> sh) ^ x1 ^ np.uint64(ka), p1 & lo, (p0 >> sh) ^ x3 ^ np.uint64(kb), p0 & lo
        ka, kb = (ka + 0x9E3779B9) % 2 ** 32, (kb + 0xBB67AE85) % 2 ** 32
    d = np.empty((rows * nb, 8), dtype=np.uint32)
    for k, word in enumerate((x0, x1, x2, x3)):
        d[:, 2 * k], d[:, 2 * k + 1] = word % np.uint64(65536), word // np.uint64(65536)
    t = int(65536 * case["p"] + 0.5)
    kept = d.reshape(rows, 8 * nb)[:, :units] >= t
    f = torch.from_numpy(kept).cuda().double() * (65536 / (65536 - t))
    return f.repeat_interleave(group, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    n, x = case["rows"], st["x"].double()
    shape = x.shape
    x = x.reshape(n, -1)
    factor = _exact_factor(case, st["seed"], st["offset"]) if case["p"] else 1.0
    if case["op"] == "dropout":
        return (x * factor).reshape(shape)
    res = st["r"].double().reshape(n, -1) if case["residual"] else 0.0
    back = case["op"].endswith("backward")
    s = x if back else x * factor + res
    # columns of each part that is normalised by itself: a whole row, or one degree
    if "channels" in case:
        l_max, ch = case["l_max"], case["channels"]
        parts = []
        for l in range(l_max + 1):
            comp = torch.arange(l * l, (l + 1) ** 2, device="cuda")
            parts.append((torch.arange(ch, device="cuda")[:, None] * (l_max + 1) ** 2 + comp).reshape(-1))
        weight = [st["w"][l].double().repeat_interleave(2 * l + 1) for l in range(l_max + 1)]
    else:
        parts, weight = [slice(None)], [st["w"].double()]
    y, dr = torch.empty_like(s), torch.empty_like(s)
    stats, dws, db = [], [], None
    g = st["g"].double().reshape(n, -1) if back else None
    for l, at in enumerate(parts):
        v = s[:, at]
        mu = v.mean(dim=1) if l == 0 else torch.zeros(n, device="cuda", dtype=torch.float64)
        if back:
            mu = st["stats"][:, 0].double() if l == 0 else mu
            q = st["stats"][:, 1 + l].double()
            hat = (v - mu[:, None]) * q[:, None]
            a = g[:, at] * weight[l]
            d = a - hat * (a * hat).mean(dim=1)[:, None]
            dr[:, at] = q[:, None] * (d - a.mean(dim=1)[:, None] if l == 0 else d)
            dws.append((g[:, at] * hat).sum(dim=0).reshape(-1, 2 * l + 1).sum(dim=1))
            if l == 0:
                db = g[:, at].sum(dim=0)
        else:
            v = v - mu[:, None]
            q = 1 / torch.sqrt((v * v).mean(dim=1) + EPS)
            y[:, at] = v * q[:, None] * weight[l] + (st["b"].double() if l == 0 else 0.0)
            stats += [mu, q] if l == 0 else [q]
    if back:
        dr = dr + res
        got = dict(x=(dr * factor).reshape(shape), w=torch.stack(dws) if "channels" in case else dws[0], b=db)
        if _apart(case):
            got["r"] = dr.reshape(shape)
        return got
    got = dict(y=y.reshape(shape), stats=torch.stack(stats, dim=1))
    if _sums(case):
        got["s"] = s.reshape(shape)
    return got


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n, d = case["rows"], _width(case)
    t = 2 if case["dtype"] == "bf16" else 4
    op, values = case["op"], case["rows"] * _width(case)
    random = values / (8 * (case.get("group") or (case["l_max"] + 1) ** 2)) * 40 if case["p"] else 0
    if op == "dropout":
        return {"bytes": 2 * values * t, "flops": values + random}
    plane = values * t
    per_row = 4 * _stats_width(case) * n
    params = 4 * (case["channels"] * (case["l_max"] + 2) if "channels" in case else 2 * d)
    if op.endswith("backward"):
        # g, s and where there is one the sum's own gradient in; dx and where it is another one the sum's out; w in, dw, db out
        planes = 3 + int(case["residual"]) + int(_apart(case))
        return {"bytes": planes * plane + per_row + 2 * params, "flops": 13 * values + random}
    planes = 2 + int(case["residual"]) + int(_sums(case))
    return {"bytes": planes * plane + per_row + params, "flops": 8 * values + random}
