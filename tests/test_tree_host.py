"""Rotary positions and drafted trees without a GPU: frequencies of the scalings, the oracle's
attention against the decode oracle, and what the entry points refuse before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4, tree

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, TIMEOUT, WORKSPACE, BAD_PAGE = range(8)
P = ctypes.c_void_p(0x10000)   # a fake, aligned "device" address (never dereferenced)
MIS = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_tmem_gb300 import build
    build.build()
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa.library()


def test_frequencies():
    import scaled_dot_product_tmem_gb300 as sdpa
    cpu = dict(device="cpu")
    w, g = sdpa.rope_frequencies(64, **cpu)
    assert g == 1.0 and w.dtype == torch.float64 and np.allclose(w.numpy(), 10000.0 ** -(np.arange(32) / 32), rtol=1e-14)
    lin, g = sdpa.rope_frequencies(64, scaling="linear", factor=8.0, **cpu)
    assert g == 1.0 and np.allclose(lin.numpy(), w.numpy() / 8, rtol=1e-14)
    b, g = sdpa.rope_frequencies(64, scaling="base", factor=8.0, **cpu)
    assert b[0] == 1.0 and math.isclose(b[-1], w[-1] / 8, rel_tol=1e-12)  # the fastest stays, the slowest is divided
    p, g = sdpa.rope_frequencies(64, scaling="parts", factor=8.0, original_length=2048, **cpu)
    assert math.isclose(g, 0.1 * math.log(8.0) + 1)
    turns = 2048 * w.numpy() / (2 * math.pi)
    r = (p / w).numpy()
    assert np.allclose(r[turns >= 32], 1.0, rtol=1e-14) and np.allclose(r[turns <= 1], 1 / 8, rtol=1e-14)
    assert np.all(np.diff(r) <= 1e-15)
    assert sdpa.rope_frequencies(64, scaling="parts", factor=8.0, original_length=64, gain=2.0, **cpu)[1] == 2.0
    for bad in (dict(rot_dim=20), dict(rot_dim=0), dict(rot_dim=512), dict(rot_dim=64, base=0.0),
                dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="parts"), dict(rot_dim=64, factor=-1.0),
                dict(rot_dim=64, factor=float("nan"))):
        with pytest.raises(ValueError):
            sdpa.rope_frequencies(**bad, **cpu)


def test_angles_of_far_positions():
    """Whole turns drop out: frequency 2 pi / 1024 at any multiple of 1024."""
    w = np.array([2 * math.pi / 1024])
    a = tree.angles([0, 1024, 1024 * 2 ** 20, 256 + 1024 * 2 ** 20], w)
    assert np.all(np.abs(a[:3]) < 1e-6) and abs(a[3, 0] - math.pi / 2) < 1e-6


def test_a_chain_is_the_decode():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((4, 4, 64))
    for w in (-1, 0, 2):
        a = tree.attention(q, k, v, 5, None, window=w, sink=np.zeros(4))
        b = kv4.decode(q, k, v, 9, window=w, sink=np.zeros(4))
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-12)
    assert tree.path([-1, 0, 0, 1, 9, -5], 3) == [3, 1, 0] and tree.path([-1, 0, 0, 1, 9], 4) == [4]


def test_rope_validation(lib):
    def table(w=P, pos=P, t=P, T=4, n=32, gain=1.0):
        return lib.attn_rope_table(w, pos, t, T, n, ctypes.c_float(gain), None)

    assert table(T=-1) == INVALID and table(n=-8) == INVALID and table(gain=float("nan")) == INVALID
    assert table(n=0) == UNSUPPORTED and table(n=12) == UNSUPPORTED and table(n=136) == UNSUPPORTED
    assert table(w=None) == INVALID and table(pos=None) == INVALID and table(t=None) == INVALID
    assert table(t=MIS) == MISALIGNED and table(w=ctypes.c_void_p(0x10004)) == MISALIGNED
    assert table(T=0, w=None) == OK

    def rope(q=P, k=P, t=P, qo=P, ko=P, T=4, H=2, Hk=1, d=64, n=32, first=0, R=4, qs=128, ks=64, qos=128, kos=64):
        return lib.attn_rope(q, k, t, qo, ko, T, H, Hk, d, n, first, R, qs, ks, qos, kos, 0, 0, None)

    assert rope(T=-1) == INVALID and rope(H=-1) == INVALID and rope(d=0) == INVALID and rope(first=-8) == INVALID
    assert rope(n=12) == UNSUPPORTED and rope(n=0) == UNSUPPORTED and rope(d=60) == UNSUPPORTED
    assert rope(first=4, n=8) == UNSUPPORTED and rope(d=264, qs=528, qos=528, ks=264, kos=264) == UNSUPPORTED
    assert rope(first=8) == INVALID                      # past the head
    assert rope(R=3) == INVALID and rope(R=0) == INVALID  # rows of the table
    assert rope(q=None) == INVALID and rope(ko=None) == INVALID and rope(t=None) == INVALID
    assert rope(qs=120) == INVALID and rope(kos=56) == INVALID
    assert rope(qs=132) == INVALID                       # q and q_out are the same: so must be their rows
    assert rope(qo=ctypes.c_void_p(0x20000), qs=132) == MISALIGNED
    assert rope(q=MIS) == MISALIGNED and rope(t=MIS) == MISALIGNED
    assert rope(T=0, q=None) == OK and rope(H=0, Hk=0, q=None, k=None) == OK


def test_append_rope_validation(lib):
    def app(q=P, k=P, v=P, t=P, qo=P, cu=P, pool=P, table=P, lens=P, B=2, T=5, H=4, Hk=2, d=128, pages=4, page=16, mp=3, n=64,
            first=0, qs=512, ks=256, vs=256, qos=512):
        return lib.attn_kv4_append_rope(q, k, v, t, qo, cu, pool, table, lens, B, T, H, Hk, d, pages, page, mp, n, first, qs,
                                        ks, vs, qos, 0, None)

    assert app(B=-1) == INVALID and app(T=-1) == INVALID and app(Hk=0) == INVALID and app(H=-1) == INVALID
    assert app(d=192) == UNSUPPORTED and app(page=24) == UNSUPPORTED and app(n=20) == UNSUPPORTED
    assert app(first=8) == INVALID and app(n=72) == INVALID
    assert app(ks=248) == INVALID and app(vs=260) == MISALIGNED and app(qs=504) == INVALID
    assert app(k=None) == INVALID and app(t=None) == INVALID and app(q=None) == INVALID and app(pool=None) == INVALID
    assert app(H=0, q=None, qo=None, t=None) == INVALID
    assert app(k=MIS) == MISALIGNED and app(q=MIS) == MISALIGNED and app(t=MIS) == MISALIGNED
    assert app(T=0) == OK and app(B=0, H=0, q=None) == OK


def test_tree_validation(lib):
    need = lib.attn_kv4_tree_workspace_size(2, 5, 8, 2, 128)
    assert need > 0
    assert lib.attn_kv4_tree_workspace_size(2, 5, 8, 3, 128) == 0 and lib.attn_kv4_tree_workspace_size(2, 5, 8, 2, 96) == 0

    def tr(q=P, cu=P, par=P, pool=P, table=P, lens=P, o=P, lse=None, B=2, T=5, H=8, Hk=2, d=128, page=16, mp=3, scale=0.0,
           window=-1, st=0, off=None, zero=0, ws=P, wsb=need):
        return lib.attn_kv4_tree(q, cu, par, pool, table, lens, o, lse, B, T, H, Hk, d, 4, page, mp, ctypes.c_float(scale),
                                 window, st, off, zero, ws, ctypes.c_size_t(wsb), None)

    assert tr(H=7) == INVALID and tr(B=-1) == INVALID and tr(T=-1) == INVALID
    assert tr(d=192) == UNSUPPORTED and tr(page=20) == UNSUPPORTED and tr(scale=2e30) == UNSUPPORTED
    assert tr(H=1 << 17, Hk=1, T=1) == UNSUPPORTED and tr(T=1 << 29) == UNSUPPORTED
    assert tr(st=3) == INVALID and tr(st=2) == INVALID
    assert tr(q=None) == INVALID and tr(o=None) == INVALID and tr(lens=None) == INVALID and tr(cu=None) == INVALID
    assert tr(pool=None) == INVALID
    assert tr(q=MIS) == MISALIGNED and tr(par=ctypes.c_void_p(0x10002)) == MISALIGNED
    assert tr(ws=None) == WORKSPACE and tr(wsb=need - 1) == WORKSPACE and tr(ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    assert tr(T=0) == OK and tr(B=0) == OK


def test_keep_validation(lib):
    def keep(pool=P, table=P, lens=P, kept=P, B=2, most=3, layers=1, H=2, d=128, pages=4, page=16, mp=3):
        return lib.attn_kv4_keep(pool, table, lens, kept, B, most, layers, H, d, pages, page, mp, None)

    assert keep(B=-1) == INVALID and keep(most=-1) == INVALID and keep(layers=-1) == INVALID and keep(H=0) == INVALID
    assert keep(d=96) == UNSUPPORTED and keep(page=8) == UNSUPPORTED and keep(B=70000) == UNSUPPORTED
    assert keep(layers=70000) == UNSUPPORTED
    assert keep(pool=None) == INVALID and keep(kept=None) == INVALID and keep(lens=None) == INVALID
    assert keep(pool=MIS) == MISALIGNED and keep(kept=ctypes.c_void_p(0x10001)) == MISALIGNED
    assert keep(B=0) == OK and keep(most=0) == OK and keep(layers=0) == OK


def test_python_refusals_without_a_gpu():
    import scaled_dot_product_tmem_gb300 as sdpa
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((4, 2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.rope_forward(q, None, t)
    with pytest.raises(ValueError):
        sdpa.rope_table(torch.zeros(32, dtype=torch.float64), torch.zeros(4, dtype=torch.int32))
    pool = torch.zeros((4, 2, sdpa.kv4_block_bytes(16, 64)), dtype=torch.uint8)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.attn_kv4_keep(pool, i32(0, 1).view(1, 2), i32(0), i32(0).view(1, 1), 64)
    with pytest.raises(ValueError):
        sdpa.sdpa_tree_kv4(q, i32(0, 4), None, pool, i32(0, 1).view(1, 2), i32(0))
