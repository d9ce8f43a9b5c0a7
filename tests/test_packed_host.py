"""Packed-sequence entry points without a GPU: workspace sizes and what they refuse before any
launch."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, TIMEOUT, WORKSPACE = range(7)
P = ctypes.c_void_p(0x10000)   # a fake, aligned "device" address (never dereferenced)
MIS = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_tmem_gb300 import build
    build.build()
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa.library()


def test_workspace_sizes(lib):
    ws = lib.attn_packed_workspace_size
    assert ws(3, 100, 100, 4, 2, 128, 128, 0) > 0
    assert ws(3, 100, 100, 4, 2, 128, 128, 1) > ws(3, 100, 100, 4, 2, 128, 128, 0)
    assert ws(0, 0, 0, 4, 2, 64, 64, 0) > 0
    assert ws(3, 100, 100, 4, 2, 192, 128, 1) > 0
    for bad in ((3, 100, 100, 4, 3, 128, 128), (-1, 100, 100, 4, 2, 128, 128), (3, 100, 100, 4, 2, 128, 64),
                (3, 100, 100, 4, 2, 96, 96), (3, 0x7fffff00, 100, 4, 2, 64, 64)):
        assert ws(*bad, 0) == 0, bad


def test_fwd_validation(lib):
    def f(q=P, k=P, v=P, o=P, lse=P, cu=P, ck=None, B=2, Tq=64, Tk=64, Hq=4, Hkv=2, dqk=128, dv=128, causal=1, window=-1,
          st=0, off=None, ws=P, wsb=1 << 20):
        return lib.attn_fwd_packed(q, k, v, o, lse, cu, ck, B, Tq, Tk, Hq, Hkv, dqk, dv, ctypes.c_float(0.0), causal,
                                   window, st, off, 0, ws, ctypes.c_size_t(wsb), None)

    assert f(Hq=3) == INVALID and f(B=-1) == INVALID and f(Tq=-1) == INVALID and f(Tk=-2) == INVALID
    assert f(st=3) == INVALID and f(st=2) == INVALID                   # learnable needs the offset
    assert f(dqk=96) == UNSUPPORTED and f(dv=64) == UNSUPPORTED and f(dqk=192, dv=192) == UNSUPPORTED
    assert f(causal=0, window=8) == UNSUPPORTED                        # window only with causal
    assert f(q=None) == INVALID and f(cu=None) == INVALID and f(k=None) == INVALID and f(lse=None) == INVALID
    assert f(q=MIS) == MISALIGNED and f(o=MIS) == MISALIGNED
    assert f(cu=ctypes.c_void_p(0x10002)) == MISALIGNED and f(ck=ctypes.c_void_p(0x10001)) == MISALIGNED
    assert f(ws=None) == WORKSPACE and f(wsb=16) == WORKSPACE and f(ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    assert f(B=0) == OK and f(Tq=0) == OK


def test_bwd_validation(lib):
    def b(q=P, dq=P, dk=P, doff=None, cu=P, B=2, Tq=64, Tk=64, Hq=4, Hkv=2, d=128, st=0, off=None, ws=P,
          wsb=1 << 24, window=-1, causal=1):
        return lib.attn_bwd_packed(q, P, P, P, P, P, dq, dk, P, doff, cu, None, B, Tq, Tk, Hq, Hkv, d, d,
                                   ctypes.c_float(0.0), causal, window, st, off, 0, ws, ctypes.c_size_t(wsb), None)

    assert b(Hq=5) == INVALID and b(B=-3) == INVALID
    assert b(st=2, off=P) == INVALID                                   # learnable needs d_offset
    assert b(causal=0, window=3) == UNSUPPORTED and b(d=192) == UNSUPPORTED
    assert b(q=None) == INVALID and b(dk=None) == INVALID and b(cu=None) == INVALID
    assert b(dq=MIS) == MISALIGNED and b(doff=ctypes.c_void_p(0x10002)) == MISALIGNED
    assert b(ws=None) == WORKSPACE and b(wsb=1024) == WORKSPACE and b(ws=ctypes.c_void_p(0x10080)) == WORKSPACE
    assert b(B=0) == OK


def test_python_refusals_without_a_gpu():
    import scaled_dot_product_tmem_gb300 as sdpa
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa._check_packed(q, q, q, cu, None, None)
    with pytest.raises(TypeError):
        sdpa._check_packed(q.float(), q, q, cu, None, None)
    with pytest.raises(ValueError):
        sdpa._check_packed(q[0], q, q, cu, None, None)
