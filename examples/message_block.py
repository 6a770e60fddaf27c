"""One residual message block trained with the library's entry points alone.

    h  = degree_norm(x)                                  node features, l <= 3
    t  = rbf W1,  a = silu(layer_norm(dropout(t))),  R = a W2     radial network
    m  = eqmp_fused(vec, h; R, M)                        messages, summed into the receivers
    y, s = degree_norm(m, residual=x, dropout by channel)         s = x + dropout(m) is the residual stream
    loss = 1/2 |y - target|^2 / N

forward() and backward() are the two halves of a step; train() runs a few of
them with plain gradient descent.  The dropout masks are never stored: both
halves are given the same Dropout.

    python examples/message_block.py [atoms] [channels] [steps]
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import equivariant_gnn_message_gb300 as eq  # noqa: E402
from equivariant_gnn_message_gb300.inputs import make_workload  # noqa: E402


def problem(n_atoms, channels, hidden=64, seed=0):
    """A graph with radial features, input features, a target, and the parameters, on the GPU."""
    wl = make_workload(n_atoms=n_atoms, cutoff=5.0, channels=channels, weights="radial", storage="f32", seed=seed)
    rng = np.random.default_rng(seed + 1)
    up = lambda a, dt=np.float32: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()  # noqa: E731
    offs, edges = eq.sender_view(wl.src, wl.n_atoms)
    graph = dict(vec=up(wl.vec), off=up(wl.off, np.int32), src=up(wl.src, np.int32), dst=up(wl.dst, np.int32),
                 send_off=up(offs, np.int32), send_edges=up(edges, np.int32), rbf=up(wl.R))
    normal = lambda *s: up(rng.standard_normal(s))  # noqa: E731
    params = dict(w1=normal(8, hidden) * 0.5, ln_w=torch.ones(hidden, device="cuda"), ln_b=torch.zeros(hidden, device="cuda"),
                  w2=normal(hidden, 8) * hidden ** -0.5, M=up(wl.M),
                  pre_w=torch.ones(4, channels, device="cuda"), pre_b=torch.zeros(channels, device="cuda"),
                  post_w=torch.ones(4, channels, device="cuda"), post_b=torch.zeros(channels, device="cuda"))
    return graph, up(wl.x), normal(wl.n_atoms, channels, 16), params


def masks(p, seed, step):
    """The two Dropouts of a step: by element in the radial network, by channel on the messages."""
    if not p:
        return None, None
    return eq.Dropout(p, seed, offset=2 * step), eq.Dropout(p, seed, offset=2 * step + 1, group=16)


def forward(graph, x, target, prm, drops):
    """The loss and what the backward half needs."""
    k = {"x": x}
    pre = eq.eqmp_degree_norm(x, prm["pre_w"], prm["pre_b"], need=("y", "stats"))
    k["h"], k["pre_stats"] = pre["y"], pre["stats"]
    hid = eq.eqmp_layer_norm(graph["rbf"] @ prm["w1"], prm["ln_w"], prm["ln_b"], drop=drops[0], need=("y", "s", "stats"))
    k["hid"] = hid
    k["a"] = torch.nn.functional.silu(hid["y"])
    k["R"] = k["a"] @ prm["w2"]
    m = eq.eqmp_fused(graph["vec"], k["h"], graph["off"], graph["src"], R=k["R"], M=prm["M"])
    k["post"] = eq.eqmp_degree_norm(m, prm["post_w"], prm["post_b"], residual=x, drop=drops[1], need=("y", "s", "stats"))
    k["gy"] = (k["post"]["y"] - target) / x.shape[0]
    return 0.5 * (k["gy"] * (k["post"]["y"] - target)).sum(), k


def backward(graph, k, prm, drops):
    """Gradients of the loss: of every parameter and of x."""
    g = {}
    post = eq.eqmp_degree_norm_backward(k["gy"], k["post"]["s"], k["post"]["stats"], prm["post_w"], drop=drops[1],
                                        need=("x", "r", "w", "b"))
    g["post_w"], g["post_b"] = post["w"], post["b"]
    msg = eq.eqmp_fused_backward(graph["vec"], k["h"], graph["off"], graph["src"], graph["dst"], graph["send_off"],
                                 graph["send_edges"], post["x"], R=k["R"], M=prm["M"], need=("x", "R", "M"))
    g["M"] = msg["M"]
    pre = eq.eqmp_degree_norm_backward(msg["x"], k["x"], k["pre_stats"], prm["pre_w"], grad_s=post["r"])
    g["x"], g["pre_w"], g["pre_b"] = pre["x"], pre["w"], pre["b"]
    g["w2"] = k["a"].t() @ msg["R"]
    u = k["hid"]["y"]
    sig = torch.sigmoid(u)
    gu = (msg["R"] @ prm["w2"].t()) * sig * (1 + u * (1 - sig))
    hid = eq.eqmp_layer_norm_backward(gu, k["hid"]["s"], k["hid"]["stats"], prm["ln_w"], drop=drops[0])
    g["ln_w"], g["ln_b"] = hid["w"], hid["b"]
    g["w1"] = graph["rbf"].t() @ hid["x"]
    return g


def train(n_atoms=1000, channels=32, steps=20, p=0.1, rate=1e-3, seed=0):
    """Gradient descent on the block's parameters; the losses without dropout before and after."""
    graph, x, target, prm = problem(n_atoms, channels, seed=seed)
    before = float(forward(graph, x, target, prm, (None, None))[0])
    for step in range(steps):
        drops = masks(p, seed + 7, step)
        _, kept = forward(graph, x, target, prm, drops)
        for name, g in backward(graph, kept, prm, drops).items():
            if name != "x":
                prm[name] -= rate * g
    return before, float(forward(graph, x, target, prm, (None, None))[0])


if __name__ == "__main__":
    import __graft_entry__

    __graft_entry__.build()
    args = [int(v) for v in sys.argv[1:]]
    print("loss %.4f -> %.4f" % train(*args))
