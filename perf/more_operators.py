"""Attention over a receiver's edges: the measured cases and their plain forms.

Operators (the framework's entry points of the same names):
  head_norm               queries and keys [N, H, D] divided by the root mean square of each head, times a weight, and
                          rotated in pairs by angles that are linear in a node's position (a place in a chain, a time,
                          or coordinates with wave vectors)
  head_norm_backward      its gradients: of the queries, the keys, the weights and the positions
  edge_bias               a learned bias of each edge and head, by the bucket of the edge's length
  edge_bias_backward      the gradient of the table: sums over the edges of each bucket
  edge_attention          softmax over a receiver's edges of scale q.k + bias, and the sum of the senders' values by it
  edge_attention_backward its gradients: of the queries, keys, values and the bias

An edge whose score is minus infinity is left out, whatever its key and value hold; a receiver that is left without an
edge gets zeros, and zeros as its statistics.  The statistics of a row are the largest score and the sum of
exp(score - largest).  bucket[e] is the number of borders that are at most |vec_e|, decided on squares in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a 64-atom molecule, one call of a small inference loop: latency; positions are places in a chain
        dict(name="head_norm_f32_64x4x16", op="head_norm", dtype="f32", nodes=64, heads=4, kheads=4, dim=16, axes=1, pad=0),
        # a 100,000-atom system in training: queries and keys cut out of one projection, rotated by coordinates
        dict(name="head_norm_bf16_100000x8x32", op="head_norm", dtype="bf16", nodes=100000, heads=8, kheads=8, dim=32,
             axes=3, pad=256),
        # an odd number of nodes and a head that no vector divides, fewer key heads, no rotation
        dict(name="head_norm_bwd_f32_4999x6x18", op="head_norm_backward", dtype="f32", nodes=4999, heads=6, kheads=2, dim=18,
             axes=0, pad=5),
        # the training step of the large system, positions with gradients (forces)
        dict(name="head_norm_bwd_f32_100000x8x32", op="head_norm_backward", dtype="f32", nodes=100000, heads=8, kheads=8,
             dim=32, axes=3, pad=0),
        # the edges of a 64-atom molecule
        dict(name="edge_bias_782x4", op="edge_bias", edges=782, heads=4, buckets=16),
        # the edges of a 100,000-atom system
        dict(name="edge_bias_1909372x8", op="edge_bias", edges=1909372, heads=8, buckets=64),
        # the gradient on the benchmark's 1000 atoms
        dict(name="edge_bias_bwd_16516x4", op="edge_bias_backward", edges=16516, heads=4, buckets=32),
        # and on the large system
        dict(name="edge_bias_bwd_1909372x8", op="edge_bias_backward", edges=1909372, heads=8, buckets=64),
        # 1000 atoms of 32 channels of degree 3, 4 heads of 8 channels: the benchmark's size, inference
        dict(name="attn_f32_1000_c32", op="edge_attention", dtype="f32", atoms=1000, cutoff=5.0, sorted=False, hub=False,
             masked=0.0, heads=4, dim=16, vdim=128, pad=0),
        # 100,000 atoms of 64 channels, 8 heads, atoms in no order: the gather at its hardest
        dict(name="attn_f32_100000_c64", op="edge_attention", dtype="f32", atoms=100000, cutoff=5.0, sorted=False, hub=False,
             masked=0.0, heads=8, dim=32, vdim=128, pad=0),
        # degree 4 with 16 channels (rows of odd lengths), masked edges and one node that is linked with all others
        dict(name="attn_bwd_f32_1000_hub", op="edge_attention_backward", dtype="f32", atoms=1000, cutoff=5.0, sorted=False,
             hub=True, masked=0.1, heads=4, dim=18, vdim=100, pad=6),
        # 10,000 atoms with a wide cutoff, 128 channels in bf16: dense, mixed precision
        dict(name="attn_bwd_bf16_10000_c128", op="edge_attention_backward", dtype="bf16", atoms=10000, cutoff=7.0,
             sorted=True, hub=False, masked=0.0, heads=8, dim=32, vdim=256, pad=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["head_norm", "head_norm_backward", "edge_bias", "edge_bias_backward", "edge_attention",
                     "edge_attention", "edge_attention_backward", "edge_attention_backward"])
    if op.startswith("edge_bias"):
        heads = rng.choice([1, 2, 3, 4, 6, 8, 8, 16])
        return dict(op=op, edges=_spread(rng, 1, 1900000 * 8 // max(heads, 8)), heads=heads, buckets=_spread(rng, 1, 256))
    dtype = rng.choice(["f32", "bf16"])
    heads = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 12, 16])
    if op.startswith("head_norm"):
        dim = rng.choice([8, 16, 32, 32, 64, 128, rng.randint(1, 64) * 2, rng.randint(1, 128) * 2])
        axes = rng.choice([0, 1, 2, 3])
        if axes == 0 and rng.random() < 0.3:
            dim -= 1
        kheads = rng.choice([heads, heads, 1, rng.randint(1, heads)])
        return dict(op=op, dtype=dtype, nodes=_spread(rng, 1, min(100000, 100000 * 512 // ((heads + kheads) * dim))),
                    heads=heads, kheads=kheads, dim=dim, axes=axes, pad=rng.choice([0, 0, 3, 64, rng.randint(1, 300)]))
    dim = rng.choice([8, 16, 32, 32, 64, 128, rng.randint(1, 80)])
    l_max = rng.choice([0, 3, 3, 3, 4, 5, 6])
    vdim = (l_max + 1) ** 2 * rng.choice([1, 2, 4, 8, 8, rng.randint(1, 12)])
    cutoff = rng.choice([4.0, 5.0, 5.0, 6.0, 7.0])
    edges_per_atom = 0.038 * 4 / 3 * math.pi * cutoff ** 3
    most = 100000 * 19 * 8 * 160 / (edges_per_atom * heads * (dim + vdim)) / 2
    return dict(op=op, dtype=dtype, atoms=_spread(rng, 2, max(3, min(100000, int(most)))), cutoff=cutoff,
                sorted=rng.random() < 0.5, hub=rng.random() < 0.25, masked=rng.choice([0.0, 0.0, 0.05, 0.5]), heads=heads,
                dim=dim, vdim=vdim, pad=rng.choice([0, 0, 0, 1, 8, rng.randint(1, 100)]))


# ------------------------------------------------------------------ inputs
def _positions(n, gen):
    """n atoms in a cube at the density of a molecular liquid."""
    side = (n / 0.038) ** (1 / 3)
    return torch.rand(n, 3, generator=gen, device="cuda") * side


def _by_cell(pos, cutoff):
    """The atoms' order along the Morton curve of their cells."""
    c = (pos / cutoff).long()
    key = sum(((c[:, a] >> bit) & 1) << (3 * bit + a) for bit in range(10) for a in range(3))
    return torch.argsort(key, stable=True)


def _pairs(pos, reach):
    """All pairs (i, j), i < j, closer than `reach`, and their squared distances."""
    n = pos.shape[0]
    cell = (pos / reach).long()
    m = int(cell.max()) + 3
    key = ((cell[:, 0] + 1) * m + cell[:, 1] + 1) * m + cell[:, 2] + 1
    key_sorted, order = torch.sort(key)
    found = []
    for dx in (-1, 0, 1):
        for dy in (-1, 0, 1):
            near = key + (dx * m + dy) * m
            first = torch.searchsorted(key_sorted, near - 1)
            count = torch.searchsorted(key_sorted, near + 1, right=True) - first
            i = torch.repeat_interleave(torch.arange(n, device="cuda"), count)
            at = torch.arange(i.shape[0], device="cuda") - (count.cumsum(0) - count)[i] + first[i]
            j = order[at]
            square = (pos[j] - pos[i]).square().sum(1)
            keep = (square < reach * reach) & (i < j)
            found.append((i[keep], j[keep], square[keep]))
    return [torch.cat(part) for part in zip(*found)]


def _pair_count(case):
    """Pairs of atoms closer than the cutoff, in the mean: for two points of a unit cube and r <= 1 the probability is
    pi r^3 (4/3 - 3/2 r + 8/(5 pi) r^2 - r^3/(6 pi))."""
    n = case["atoms"]
    r = min(case["cutoff"] / (n / 0.038) ** (1 / 3), 1.0)
    near = math.pi * r ** 3 * (4 / 3 - 1.5 * r + 1.6 / math.pi * r ** 2 - r ** 3 / (6 * math.pi))
    return int(round(n * (n - 1) / 2 * near))


def _graph(case, gen):
    n = case["atoms"]
    pos = _positions(n, gen)
    if case["sorted"]:
        pos = pos[_by_cell(pos, case["cutoff"])]
    # the closest pairs, as many as the cutoff has in the mean: a batch of this size has them, whatever the seed
    side = float((n / 0.038) ** (1 / 3))
    i, j, square = _pairs(pos, 1.1 * case["cutoff"] if n > 2000 else 2 * side)
    closest = torch.argsort(square, stable=True)[:_pair_count(case)]
    i, j = i[closest], j[closest]
    dst, src = torch.cat((i, j)), torch.cat((j, i))
    both = torch.sort(dst * n + src)[0]
    dst, src = both // n, both % n
    if case["hub"]:  # one more node, linked with all others both ways
        all_, hub = torch.arange(n, device="cuda"), torch.full((n,), n, device="cuda")
        dst, src = torch.cat((dst, all_, hub)), torch.cat((src, hub, all_))
        n += 1
        both = torch.sort(dst * n + src)[0]
        dst, src = both // n, both % n
    ids = torch.arange(n + 1, device="cuda")
    order = torch.argsort(src, stable=True)
    return n, dict(off=torch.searchsorted(dst, ids).int(), src=src.int(), dst=dst.int(),
                   send_off=torch.searchsorted(src[order], ids).int(), send_edges=order.int())


def _slice(n, widths, pad, dtype, gen):
    """Tensors [n, heads, dim] cut out of one projection with `pad` other columns behind them."""
    whole = torch.randn(n, sum(h * d for h, d in widths) + pad, generator=gen, device="cuda").to(dtype)
    out, at = [], 0
    for h, d in widths:
        out.append(whole[:, at:at + h * d].unflatten(1, (h, d)))
        at += h * d
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    op, st = case["op"], dict(case=case, out={})
    if op.startswith("edge_bias"):
        E, H, B = case["edges"], case["heads"], case["buckets"]
        # lengths as neighbours have them, up to a cutoff of 7; linear borders up to 4, then in equal ratios
        r = 7 * torch.rand(E, 1, generator=gen, device="cuda") ** (1 / 3)
        vec = normal(E, 3)
        st["vec"] = vec / vec.norm(dim=1, keepdim=True) * r
        half = (B - 1) // 2
        st["borders"] = torch.cat((torch.arange(1, half + 1, device="cuda") * (4 / max(half, 1)),
                                   4 * (7 / 4) ** (torch.arange(1, B - half, device="cuda") / max(B - half, 1)))).float()
        if op == "edge_bias":
            st["table"] = normal(B, H)
            st["out"] = dict(bias=torch.empty(E, H, device="cuda"), bucket=torch.empty(E, device="cuda", dtype=torch.int32))
        else:
            st["bucket"], st["g"] = _bucket(st["vec"], st["borders"]), normal(E, H)
            st["out"] = dict(table=torch.empty(B, H, device="cuda"))
        return st
    dt = TYPES[case["dtype"]]
    if op.startswith("head_norm"):
        n, H, K, D, A = (case[k] for k in ("nodes", "heads", "kheads", "dim", "axes"))
        st["q"], st["k"] = _slice(n, ((H, D), (K, D)), case["pad"], dt, gen)
        st["wq"], st["wk"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        st["pos"] = st["freq"] = None
        if A == 1:  # places in a chain, and rates from one radian a place down in equal ratios
            st["pos"] = torch.arange(n, device="cuda").float()[:, None]
            st["freq"] = (10000.0 ** (-torch.arange(D // 2, device="cuda").float() / (D // 2)))[:, None]
        elif A:  # coordinates, and wave vectors of lengths from 2 pi / 1 down to 2 pi / 30
            st["pos"] = _positions(n, gen)[:, :A].contiguous()
            way = normal(D // 2, A)
            st["freq"] = way / way.norm(dim=1, keepdim=True) * (
                2 * math.pi * 30 ** (-torch.arange(D // 2, device="cuda") / (D // 2)))[:, None]
        new = lambda h: torch.empty(n, h, D, device="cuda", dtype=dt)  # noqa: E731
        st["out"] = dict(q=new(H), k=new(K))
        if op == "head_norm":
            st["out"]["rstd"] = torch.empty(n, H + K, device="cuda")
            st["need"] = ("q", "k", "rstd")
        else:
            st["gq"], st["gk"] = normal(n, H, D).to(dt), normal(n, K, D).to(dt)
            both = torch.cat((st["q"], st["k"]), 1).double()
            st["rstd"] = (1 / torch.sqrt(both.square().mean(2) + EPS)).float()
            st["need"] = ("q", "k", "wq", "wk") + (("pos",) if A else ())
        return st
    H, D, V = case["heads"], case["dim"], case["vdim"]
    n, graph = _graph(case, gen)
    E = graph["src"].shape[0]
    st.update(graph, n=n)
    st["q"], st["k"], st["v"] = _slice(n, ((H, D), (H, D), (H, V)), case["pad"], dt, gen)
    st["bias"] = normal(E, H)
    if case["masked"]:  # padding or a smaller cutoff: some edges do not count, and some receivers keep none
        off = torch.rand(E, generator=gen, device="cuda") < case["masked"]
        off |= (torch.rand(n, generator=gen, device="cuda") < 0.02)[graph["dst"].long()]
        st["bias"][off] = -math.inf
    new = lambda d: torch.empty(n, H, d, device="cuda", dtype=dt)  # noqa: E731
    if op == "edge_attention":
        st["out"] = dict(out=new(V), stats=torch.empty(n, H, 2, device="cuda"))
    else:
        st["g"] = normal(n, H, V).to(dt)
        st["stats"] = _row_stats(_scores(st), st)
        st["out"] = dict(q=new(D), k=new(D), v=new(V), bias=torch.empty(E, H, device="cuda"))
    return st


# ------------------------------------------------------------------ plain forms
def _bucket(vec, borders):
    """In 64 bits, where the squares of the parts are exact: a length next to a border falls on its side."""
    x, y, z = vec.double().unbind(1)
    return torch.bucketize((x * x + y * y) + z * z, borders.double().square(), right=True).int()


def _turn(st):
    """Cosine and sine [N, 1, D/2] of each node's angles, formed in 64 bits: far positions turn many times."""
    if st["pos"] is None:
        return None
    angle = (st["pos"].double()[:, None, :] * st["freq"].double()).sum(2)[:, None, :]
    return angle.cos().float(), angle.sin().float()


def _rotated(u, turn, back=False):
    if turn is None:
        return u
    c, s = turn
    s = -s if back else s
    a, b = u[:, :, 0::2], u[:, :, 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), 3).flatten(2)


def _plain_head_norm(st):
    got, turn, rstds = {}, _turn(st), []
    for name in ("q", "k"):
        x = st[name].float()
        rstd = 1 / torch.sqrt(x.square().mean(2) + EPS)
        got[name] = _rotated(x * rstd[:, :, None] * st["w" + name], turn).to(st[name].dtype)
        rstds.append(rstd)
    got["rstd"] = torch.cat(rstds, 1)
    return got


def _plain_head_norm_backward(st):
    got, turn, dpos = {}, _turn(st), 0.0
    H = st["q"].shape[1]
    for name, rstd in (("q", st["rstd"][:, :H]), ("k", st["rstd"][:, H:])):
        x, g, w = st[name].float(), st["g" + name].float(), st["w" + name]
        h = x * rstd[:, :, None]
        if turn is not None:
            y = _rotated(h * w, turn)
            dtheta = (g[:, :, 1::2] * y[:, :, 0::2] - g[:, :, 0::2] * y[:, :, 1::2]).sum(1)
            dpos = dpos + (dtheta[:, :, None] * st["freq"]).sum(1)
        g = _rotated(g, turn, back=True)
        a = g * w
        got[name] = (rstd[:, :, None] * (a - h * (a * h).mean(2, keepdim=True))).to(st[name].dtype)
        got["w" + name] = (g * h).sum((0, 1))
    if turn is not None:
        got["pos"] = dpos
    return got


def _scores(st):
    """[E, H] in 32 bits."""
    q, k = st["q"].float(), st["k"].float()
    s = (q[st["dst"].long()] * k[st["src"].long()]).sum(2) * q.shape[2] ** -0.5 + st["bias"]
    return torch.where(st["bias"] == -math.inf, -math.inf, s)


def _row_stats(s, st):
    """[N, H, 2]: the largest score of a row and the sum of exp(score - largest); zeros where nothing counts."""
    n, H = st["n"], s.shape[1]
    at = st["dst"].long()[:, None].expand(-1, H)
    m = torch.full((n, H), -math.inf, device="cuda").scatter_reduce_(0, at, s, "amax")
    m = torch.where(m == -math.inf, 0.0, m)
    z = torch.zeros(n, H, device="cuda").scatter_add_(0, at, torch.exp(s - m[st["dst"].long()]))
    return torch.stack((m, z), 2)


def _weights(s, stats, st):
    """[E, H]: the softmax over each row."""
    m, z = stats[st["dst"].long()].unbind(2)
    return torch.where(s == -math.inf, 0.0, torch.exp(s - m) / z)


def _sum_by(index, values, n):
    return torch.zeros((n,) + values.shape[1:], device="cuda").index_add_(0, index, values)


def _plain_attention(st):
    s = _scores(st)
    stats = _row_stats(s, st)
    p = _weights(s, stats, st)
    out = _sum_by(st["dst"], p[:, :, None] * st["v"].float()[st["src"].long()], st["n"])
    return dict(out=out.to(st["v"].dtype), stats=stats)


def _plain_attention_backward(st):
    dt, n, scale = st["q"].dtype, st["n"], st["q"].shape[2] ** -0.5
    src, dst = st["src"].long(), st["dst"].long()
    p = _weights(_scores(st), st["stats"], st)
    g = st["g"].float()[dst]
    dv = _sum_by(src, p[:, :, None] * g, n)
    dp = (g * st["v"].float()[src]).sum(2)
    del g
    ds = p * (dp - _sum_by(dst, p * dp, n)[dst])
    dq = _sum_by(dst, ds[:, :, None] * st["k"].float()[src], n) * scale
    dk = _sum_by(src, ds[:, :, None] * st["q"].float()[dst], n) * scale
    return dict(q=dq.to(dt), k=dk.to(dt), v=dv.to(dt), bias=ds)


def run(st):
    op = st["case"]["op"]
    if own:
        import equivariant_gnn_message_gb300 as eq

        if op == "head_norm":
            return eq.eqmp_head_norm(st["q"], st["k"], st["wq"], st["wk"], eps=EPS, pos=st["pos"], freq=st["freq"],
                                     need=st["need"], out=st["out"])
        if op == "head_norm_backward":
            return eq.eqmp_head_norm_backward(st["gq"], st["gk"], st["q"], st["k"], st["rstd"], st["wq"], st["wk"],
                                              pos=st["pos"], freq=st["freq"], need=st["need"], out=st["out"])
        if op == "edge_bias":
            return eq.eqmp_edge_bias(st["vec"], st["borders"], st["table"], need=("bias", "bucket"), out=st["out"])
        if op == "edge_bias_backward":
            return eq.eqmp_edge_bias_backward(st["g"], st["bucket"], st["case"]["buckets"], out=st["out"])
        if op == "edge_attention":
            return eq.eqmp_edge_attention(st["q"], st["k"], st["v"], st["off"], st["src"], bias=st["bias"],
                                          need=("out", "stats"), out=st["out"])
        return eq.eqmp_edge_attention_backward(st["g"], st["q"], st["k"], st["v"], st["stats"], st["off"], st["src"],
                                               st["dst"], st["send_off"], st["send_edges"], bias=st["bias"],
                                               need=("q", "k", "v", "bias"), out=st["out"])
    if op == "head_norm":
        return _plain_head_norm(st)
    if op == "head_norm_backward":
        return _plain_head_norm_backward(st)
    if op == "edge_bias":
        bucket = _bucket(st["vec"], st["borders"])
        return dict(bias=st["table"][bucket.long()], bucket=bucket)
    if op == "edge_bias_backward":
        return dict(table=_sum_by(st["bucket"], st["g"], st["case"]["buckets"]))
    return _plain_attention(st) if op == "edge_attention" else _plain_attention_backward(st)


# ------------------------------------------------------------------ in 64 bits
def _exact_head_norm(st, back):
    got, f64 = {}, torch.float64
    n, H, D = st["q"].shape
    if st["pos"] is None:
        z = torch.ones(n, 1, 1, device="cuda", dtype=torch.complex128)
    else:
        z = torch.exp(1j * (st["pos"].to(f64) @ st["freq"].to(f64).t()))[:, None, :]
    rstds, dpos = [], torch.zeros(n, st["pos"].shape[1] if st["pos"] is not None else 1, device="cuda", dtype=f64)

    def turned(u, by):  # pairs as complex numbers
        if st["pos"] is None:
            return u
        return torch.view_as_real(torch.view_as_complex(u.reshape(n, -1, D // 2, 2).contiguous()) * by).reshape(u.shape)

    for name in ("q", "k"):
        x, w = st[name].to(f64), st["w" + name].to(f64)
        r = torch.rsqrt((x * x).sum(2) / D + EPS)
        if not back:
            rstds.append(r)
            got[name] = turned(x * r.unsqueeze(2) * w, z)
            continue
        r = (st["rstd"][:, :H] if name == "q" else st["rstd"][:, H:]).to(f64).unsqueeze(2)
        g = st["g" + name].to(f64)
        gb, u = turned(g, z.conj()), x * r
        got["w" + name] = torch.einsum("nhd,nhd->d", gb, u)
        got[name] = r * (gb * w - u * torch.einsum("nhd,nhd->nh", gb * w, u).unsqueeze(2) / D)
        if st["pos"] is not None:
            # the angle turns a pair y into i y: its derivative is the real part of conj(g) i y
            y = torch.view_as_complex((u * w).reshape(n, -1, D // 2, 2).contiguous()) * z
            gc = torch.view_as_complex(g.reshape(n, -1, D // 2, 2).contiguous())
            dpos += (gc.conj() * 1j * y).real.sum(1) @ st["freq"].to(f64)
    if back and st["pos"] is not None:
        got["pos"] = dpos
    if not back:
        got["rstd"] = torch.cat(rstds, 1)
    return got


def _exact_attention(st, back):
    """One head after the other; rows are summed by differences of positions in the sorted edge list."""
    n, H, D = st["q"].shape
    src, dst = st["src"].long(), st["dst"].long()
    scale, f64 = 1 / math.sqrt(D), torch.float64
    parts = {k: [] for k in (("q", "k", "v", "bias") if back else ("out", "stats"))}
    for h in range(H):
        q, k, v, b = (st[name][:, h].to(f64) for name in ("q", "k", "v", "bias"))
        live = b != -math.inf
        i, j = dst[live], src[live]
        s = torch.einsum("ed,ed->e", q[i], k[j]) * scale + b[live]
        if back:
            m, z = st["stats"][:, h].to(f64).unbind(1)
        else:
            m = torch.zeros(n, device="cuda", dtype=f64).index_reduce_(0, i, s, "amax", include_self=False)
            z = torch.zeros(n, device="cuda", dtype=f64).index_add_(0, i, (s - m[i]).exp())
        p = (s - m[i]).exp() / z[i]
        add = lambda at, x: torch.zeros(n, x.shape[1], device="cuda", dtype=f64).index_add_(0, at, x)  # noqa: E731
        if not back:
            parts["out"].append(add(i, v[j] * p.unsqueeze(1)))
            parts["stats"].append(torch.stack((m, z), 1))
            continue
        g = st["g"][:, h].to(f64)[i]
        parts["v"].append(add(j, g * p.unsqueeze(1)))
        dp = torch.einsum("ed,ed->e", g, v[j])
        del g
        ds = p * (dp - torch.zeros(n, device="cuda", dtype=f64).index_add_(0, i, p * dp)[i])
        parts["q"].append(add(i, k[j] * (ds * scale).unsqueeze(1)))
        parts["k"].append(add(j, q[i] * (ds * scale).unsqueeze(1)))
        parts["bias"].append(torch.zeros(dst.shape[0], device="cuda", dtype=f64).masked_scatter_(live, ds))
    return {name: torch.stack(x, 1) for name, x in parts.items()}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("head_norm"):
        return _exact_head_norm(st, op.endswith("backward"))
    if op.startswith("edge_attention"):
        return _exact_attention(st, op.endswith("backward"))
    if op == "edge_bias_backward":
        table = torch.zeros(case["buckets"], case["heads"], device="cuda", dtype=torch.float64)
        for b in range(case["buckets"]):
            table[b] = st["g"][st["bucket"] == b].double().sum(0)
        return dict(table=table)
    v = st["vec"].double()
    square = (v[:, 0] ** 2 + v[:, 1] ** 2) + v[:, 2] ** 2
    bucket = torch.zeros(case["edges"], device="cuda", dtype=torch.int32)
    for b in st["borders"].double().tolist():
        bucket += square >= b * b
    return dict(bias=st["table"].double()[bucket.long()], bucket=bucket)


# ------------------------------------------------------------------ what a pass cannot do without
def _edges(case):
    return 2 * _pair_count(case) + (2 * case["atoms"] if case["hub"] else 0)


def work(case):
    op = case["op"]
    if op.startswith("edge_bias"):
        E, H, B = case["edges"], case["heads"], case["buckets"]
        if op == "edge_bias":  # vec in, the bias and the buckets out
            return {"bytes": 12 * E + 4 * E * (H + 1) + 4 * B * (H + 1), "flops": 5 * E + E * math.ceil(math.log2(B + 1))}
        return {"bytes": 4 * E * (H + 1) + 4 * B * H, "flops": E * H}
    t = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("head_norm"):
        n, heads, D, A = case["nodes"], case["heads"] + case["kheads"], case["dim"], case["axes"]
        back = op.endswith("backward")
        small = n * (4 * heads + 4 * A * (1 + back)) + 8 * D * (1 + back) + 2 * D * A
        return {"bytes": (3 if back else 2) * n * heads * D * t + small, "flops": (16 if back else 8) * n * heads * D}
    n, H, D, V = case["atoms"] + case["hub"], case["heads"], case["dim"], case["vdim"]
    E = _edges(case)
    if op == "edge_attention":
        return {"bytes": t * n * H * (2 * D + 2 * V) + 4 * E * (H + 1) + n * (4 + 8 * H), "flops": E * H * (2 * D + 2 * V + 8)}
    # q, k, v, the upstream gradient in, three gradients out; the bias in, its gradient out; the graph both ways
    return {"bytes": t * n * H * (4 * D + 3 * V) + 4 * E * (2 * H + 3) + n * (8 + 8 * H),
            "flops": E * H * (6 * D + 2 * D + 4 * V + 12)}
