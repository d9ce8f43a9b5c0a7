"""Drafted trees where each of the kernel's forms works out rows and nodes by code of its own: sinks with a
logit of their own for every head, in whole and in split segments, and trees of several units of nodes given by
their parents, also among many single tokens.  The bounds are those of test_tree_gpu.py."""
import numpy as np
import pytest
import torch

from test_tree_gpu import Trees, _clean

pytestmark = pytest.mark.gpu

GROUPS = [1, 2, 4, 14, 40]  # heads a kv head: 8, 16, 32, 128 and more rows a sequence on average


def _logits(H):
    """One of its own for every head, between -3 and 5, in no order."""
    return torch.linspace(-3.0, 5.0, H)[torch.randperm(H, generator=torch.Generator().manual_seed(H))].cuda()


@pytest.mark.parametrize("window", [-1, 700])
@pytest.mark.parametrize("sink", ["off_by_one", "learnable"])
@pytest.mark.parametrize("G", GROUPS)
def test_sinks_of_split_segments(G, sink, window):
    """A prefix whose units several CTAs share (the join ends its rows) beside short ones (some whole in a CTA)."""
    lens, nodes, Hk = [2900, 3, 0, 130], [9, 8, 7, 8], 2
    t = Trees(lens, nodes, G * Hk, Hk, 64 if window < 0 else 128, 32, seed=G)
    off = _logits(G * Hk) if sink == "learnable" else None
    o, lse = t.call(softmax_type=sink, softmax_offset=off, window=window)
    _clean()
    t.check(o, lse, window=window, sink=np.zeros(G * Hk) if off is None else off.double().cpu().numpy())


@pytest.mark.parametrize("G", GROUPS)
def test_sinks_of_whole_segments(G):
    """More short sequences than CTAs: most segments are whole, the tile's or the few rows' own code ends their rows."""
    rng = np.random.default_rng(G)
    B, Hk = 330, 2
    lens, nodes = rng.integers(0, 200, B).tolist(), rng.integers(5, 9, B).tolist()
    H = G * Hk
    t = Trees(lens, nodes, H, Hk, 64, 64, seed=G)
    off = _logits(H)
    o, lse = t.call(softmax_type="learnable", softmax_offset=off, scale=0.3)
    _clean()
    picked = rng.permutation(B)[:max(4, 80 // G)].tolist()  # (the oracle is slow)
    at, cu = t.at, t.cu
    for b in picked:
        t.lens, t.at, t.cu = [lens[b]], at[b:b + 2], cu[b:b + 2]
        t.check(o, lse, sink=off.double().cpu().numpy(), scale=float(np.float32(0.3)))


def _far_parents(rng, n):
    """Parents anywhere among the earlier nodes, a few of them roots."""
    return [int(rng.integers(-1, i)) if i % 29 else -1 for i in range(n)]


@pytest.mark.parametrize("window", [-1, 3, 200])
@pytest.mark.parametrize("kind", ["far", "chain"])
@pytest.mark.parametrize("nodes,G,singles", [([150, 300], 1, 0), ([513], 1, 0), ([300, 129], 4, 0), ([150], 7, 0),
                                             ([150], 1, 40), ([300], 1, 60), ([257, 3], 4, 200), ([140], 7, 20)])
def test_trees_of_several_units_of_nodes(nodes, G, singles, kind, window):
    """Ancestors several units above their node; row blocks far into a tree; windows that end a walk units up."""
    rng = np.random.default_rng(sum(nodes) + G)
    lens = [70, 500][:len(nodes)] + rng.integers(0, 90, singles).tolist()
    all_nodes = nodes + [1] * singles
    Hk, d = 2, 128 if G == 4 else 64
    t = Trees(lens, all_nodes, G * Hk, Hk, d, 16 if singles else 64, seed=len(lens))
    one = (lambda n: _far_parents(rng, n)) if kind == "far" else lambda n: list(range(-1, n - 1))
    t.par = [a for n in all_nodes for a in one(n)]
    o, lse = t.call(window=window)
    _clean()
    t.check(o, lse, window=window)
    if kind == "chain":  # the same without parents, by the other branch
        t.par = None
        o, lse = t.call(window=window)
        _clean()
        t.check(o, lse, window=window)
