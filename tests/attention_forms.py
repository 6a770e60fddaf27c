"""Graphs large enough for every form of the attention's kernels, and the kernels that a call launches."""
import ctypes
import re

import numpy as np

# Vectors of a key and of a value -> vectors a lane, for eight lanes a head and for sixteen; the last are ragged.
LANES8 = {(5, 7): (1, 1), (8, 13): (1, 2), (3, 27): (1, 4), (11, 30): (2, 4), (16, 61): (2, 8)}
LANES16 = {(13, 16): (1, 1), (16, 25): (1, 2), (9, 61): (1, 4), (29, 64): (2, 4), (20, 100): (2, 8)}
FEW = {(7, 15): (1, 2), (15, 61): (2, 8)}


def cases():
    """name -> (heads, head size, value size, type, receivers, what the kernels have to be: vector bytes, lanes, vectors a lane of
    key and value, rows a warp (None: not a ring))."""
    found = {}
    for dtype, size in (("f32", 4), ("bf16", 2)):
        def add(heads, key, value, vec, rows, lanes, per_lane, each):
            per = max(vec // size, 1)
            found[f"{dtype}_{vec}B_{lanes}_{per_lane[0]}_{per_lane[1]}_{each or 'any'}"] = (  # noqa: B023
                heads, key * per, value * per, dtype, rows, (vec if each else 1, lanes) + per_lane, each)  # noqa: B023

        for (k, v), per_lane in LANES8.items():
            add(4, k, v, 16, 2500, 8, per_lane, 1)
        for (k, v), per_lane in LANES16.items():
            add(2, k, v, 16, 2500, 16, per_lane, 1)
        for vec in (8, 4):
            for (k, v), per_lane in FEW.items():
                add(4, k, v, vec, 2500, 8, per_lane, 1)
        for rows, each in ((2501, 2), (3701, 3), (4903, 4)):  # a last warp of fewer rows
            add(32, 1, 3, 16, rows, 8, (1, 1), each)
        for vec in (8, 4):
            add(32, 1, 3, vec, 4903, 8, (1, 2), 4)
    found["bf16_2B_8_4_16_any"] = (4, 7, 49, "bf16", 2500, (1, 8, 4, 16), None)
    return found


def problem(eq, name):
    """Short rows, empty ones, two long ones among them, a sender of many edges, some edges masked."""
    import torch

    from tests.test_gpu_attention import Problem

    heads, dim, vdim, dtype, rows, _, _ = cases()[name]
    rng = np.random.default_rng(rows)
    degrees = rng.integers(0, 7, rows)
    mid = rows // 2
    degrees[[3, mid, mid + 1, mid + 2, rows - 1]] = [70, 700, 0, 300, 129]
    p = Problem(heads, dim, vdim, dtype, [int(d) for d in degrees], masked=0.1, seed=rows)
    p.src[rng.choice(len(p.src), 400, replace=False)] = rows - 3
    off, edges = eq.sender_view(p.src, rows)
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    p.graph, p.senders = (p.graph[0], up(p.src)), (p.senders[0], up(off), up(edges))
    return p


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS of the driver
    _fields_ = ([("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "shared")] +
                [(n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")])


def kernels(run):
    """(mangled name, CTAs along x) of the kernels that run() launches, from a graph recorded of it."""
    import torch

    cuda = ctypes.CDLL("libcuda.so.1")
    tape = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(tape):
        run()
    graph, count, found = ctypes.c_void_p(tape.raw_cuda_graph()), ctypes.c_size_t(0), []
    assert cuda.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cuda.cuGraphGetNodes(graph, nodes, ctypes.byref(count)) == 0
    for node in nodes:
        kind, at, name = ctypes.c_int(-1), _KernelNode(), ctypes.c_char_p()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(at)) == 0
            assert cuda.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(at.func)) == 0
            found.append((name.value.decode(), at.gx))
    return found


def forms(run):
    """pass -> (a ring or not, numbers of its form, CTAs along x)."""
    found = {}
    for name, ctas in kernels(run):
        m = re.search(r"k_attn_(?:bwd_)?(fwd|recv|send)(_ring)?I(?:f|13__nv_bfloat16)((?:Li\d+E)+)", name)
        if m:
            found[m[1]] = (bool(m[2]), tuple(int(n) for n in re.findall(r"Li(\d+)E", m[3]))[:4], ctas)
    return found
