"""One residual attention block trained with the library's entry points alone.

    h = degree_norm(x)                                    node features, l <= 3
    q, k = head_norm(h_0 W)                               queries and keys from the invariant (l = 0) values of h, each head
                                                          normed, and rotated by the atom's place in its chain
    b = edge_bias(vec; table)                             a learned bias by the bucket of the distance
    a = edge_attention(q, k, h; b)                        softmax over a receiver's edges, sum of the senders' features
    y, s = degree_norm(a, residual=x)
    loss = 1/2 |y - target|^2 / N

The weights of the sum are invariant, so a turns with the frame as h does.
forward() and backward() are the two halves of a step; train() runs a few of
them with plain gradient descent.

    python examples/attention_block.py [atoms] [channels] [heads] [steps]
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import equivariant_gnn_message_gb300 as eq  # noqa: E402
from equivariant_gnn_message_gb300.inputs import make_workload  # noqa: E402

HEAD = 8  # values of a query


def problem(n_atoms, channels, heads, buckets=16, seed=0):
    """A graph, input features, a target, and the parameters, on the GPU."""
    wl = make_workload(n_atoms=n_atoms, cutoff=5.0, channels=channels, weights="shared", storage="f32", seed=seed)
    rng = np.random.default_rng(seed + 1)
    up = lambda a, dt=np.float32: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()  # noqa: E731
    offs, edges = eq.sender_view(wl.src, wl.n_atoms)
    graph = dict(vec=up(wl.vec), off=up(wl.off, np.int32), src=up(wl.src, np.int32), dst=up(wl.dst, np.int32),
                 send_off=up(offs, np.int32), send_edges=up(edges, np.int32), borders=up(np.linspace(1.0, 5.0, buckets - 1)),
                 place=up(np.arange(wl.n_atoms)[:, None]), rates=up(10000.0 ** (-np.arange(HEAD // 2) / (HEAD // 2)))[:, None])
    normal = lambda *s: up(rng.standard_normal(s))  # noqa: E731
    params = dict(W=normal(channels, 2 * heads * HEAD) * channels ** -0.5, wq=torch.ones(HEAD, device="cuda"),
                  wk=torch.ones(HEAD, device="cuda"), table=normal(buckets, heads) * 0.1,
                  pre_w=torch.ones(4, channels, device="cuda"), pre_b=torch.zeros(channels, device="cuda"),
                  post_w=torch.ones(4, channels, device="cuda"), post_b=torch.zeros(channels, device="cuda"))
    return graph, up(wl.x), normal(wl.n_atoms, channels, 16), params


def forward(graph, x, target, prm):
    """The loss and what the backward half needs."""
    n, heads = x.shape[0], prm["table"].shape[1]
    k = {"x": x}
    pre = eq.eqmp_degree_norm(x, prm["pre_w"], prm["pre_b"], need=("y", "stats"))
    k["h"], k["pre_stats"] = pre["y"], pre["stats"]
    k["h0"] = k["h"][:, :, 0].contiguous()
    both = (k["h0"] @ prm["W"]).view(n, 2 * heads, HEAD)
    k["q"], k["k"] = both[:, :heads], both[:, heads:]
    k["turn"] = dict(pos=graph["place"], freq=graph["rates"])
    k["normed"] = eq.eqmp_head_norm(k["q"], k["k"], prm["wq"], prm["wk"], need=("q", "k", "rstd"), **k["turn"])
    k["bias"] = eq.eqmp_edge_bias(graph["vec"], graph["borders"], prm["table"])
    k["v"] = k["h"].view(n, heads, -1)
    k["att"] = eq.eqmp_edge_attention(k["normed"]["q"], k["normed"]["k"], k["v"], graph["off"], graph["src"],
                                      bias=k["bias"]["bias"], need=("out", "stats"))
    k["post"] = eq.eqmp_degree_norm(k["att"]["out"].view(x.shape), prm["post_w"], prm["post_b"], residual=x,
                                    need=("y", "s", "stats"))
    k["gy"] = (k["post"]["y"] - target) / n
    return 0.5 * (k["gy"] * (k["post"]["y"] - target)).sum(), k


def backward(graph, k, prm):
    """Gradients of the loss: of every parameter and of x."""
    g, heads = {}, prm["table"].shape[1]
    post = eq.eqmp_degree_norm_backward(k["gy"], k["post"]["s"], k["post"]["stats"], prm["post_w"], need=("x", "w", "b"))
    g["post_w"], g["post_b"] = post["w"], post["b"]
    att = eq.eqmp_edge_attention_backward(post["x"].view(k["v"].shape), k["normed"]["q"], k["normed"]["k"], k["v"],
                                          k["att"]["stats"], graph["off"], graph["src"], graph["dst"], graph["send_off"],
                                          graph["send_edges"], bias=k["bias"]["bias"], need=("q", "k", "v", "bias"))
    g["table"] = eq.eqmp_edge_bias_backward(att["bias"], k["bias"]["bucket"], prm["table"].shape[0])["table"]
    both = torch.empty(k["q"].shape[0], 2 * heads, HEAD, device="cuda")
    norm = eq.eqmp_head_norm_backward(att["q"], att["k"], k["q"], k["k"], k["normed"]["rstd"], prm["wq"], prm["wk"], **k["turn"])
    both[:, :heads], both[:, heads:] = norm["q"], norm["k"]
    both = both.flatten(1)
    g["wq"], g["wk"], g["W"] = norm["wq"], norm["wk"], k["h0"].t() @ both
    gh = att["v"].view(k["x"].shape)
    gh[:, :, 0] += both @ prm["W"].t()
    pre = eq.eqmp_degree_norm_backward(gh, k["x"], k["pre_stats"], prm["pre_w"], grad_s=post["x"])
    g["x"], g["pre_w"], g["pre_b"] = pre["x"], pre["w"], pre["b"]
    return g


def train(n_atoms=1000, channels=32, heads=4, steps=20, rate=1e-3, seed=0):
    """Gradient descent on the block's parameters; the losses before and after."""
    graph, x, target, prm = problem(n_atoms, channels, heads, seed=seed)
    before = float(forward(graph, x, target, prm)[0])
    for _ in range(steps):
        _, kept = forward(graph, x, target, prm)
        for name, g in backward(graph, kept, prm).items():
            if name != "x":
                prm[name] -= rate * g
    return before, float(forward(graph, x, target, prm)[0])


if __name__ == "__main__":
    import __graft_entry__

    __graft_entry__.build()
    print("loss %.4f -> %.4f" % train(*[int(v) for v in sys.argv[1:]]))
