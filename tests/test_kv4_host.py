"""The 4-bit paged cache without a GPU: the number format's error bounds, where a page keeps
its bytes, and what the entry points refuse before any launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, TIMEOUT, WORKSPACE, BAD_PAGE = range(8)
P = ctypes.c_void_p(0x10000)   # a fake, aligned "device" address (never dereferenced)
MIS = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_tmem_gb300 import build
    build.build()
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa.library()


def test_held_values_error_bound_and_exactness():
    """|x - held| <= s / 2 with s <= max|x| / 7 * 17/16 while the scale is a normal number, and
    held values are bf16 numbers."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((200, 128)) * 10.0 ** rng.uniform(-3, 4, (200, 1))).to(torch.bfloat16)
    xd = x.double().numpy()
    c, b = kv4.quantise(xd)
    h = kv4.values(c, b)
    s = kv4.SCALES[b]
    amax = np.abs(xd.reshape(200, 8, 16)).max(-1)
    normal = (amax / 7 >= 2.0 ** -14)
    assert normal.all()
    assert np.all(np.abs(s - amax / 7) <= amax / 7 / 16)      # 4 significant bits: half a step is 2^-4
    err = np.abs(h - xd).reshape(200, 8, 16)
    assert np.all(err <= s[..., None] / 2 + 1e-12 * amax[..., None])
    assert np.array_equal(torch.from_numpy(h).to(torch.bfloat16).double().numpy(), h)
    assert c.min() >= 0 and c.max() <= 15


def test_scale_format_is_a_truncated_half():
    byts = np.arange(0xF8)
    half = (byts.astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(half, kv4.SCALES)
    assert np.isnan((np.array([0xFF], np.uint16) << 7).view(np.float16))[0]
    assert np.array_equal(kv4.scale_bytes(kv4.SCALES), byts)          # every scale is its own nearest
    assert kv4.scale_bytes([1e9])[0] == 0xF7 and kv4.scale_bytes([0.0])[0] == 0
    mid = (kv4.SCALES[:-1] + kv4.SCALES[1:]) / 2
    assert np.all(kv4.scale_bytes(mid) % 2 == 0)                      # ties go to the even byte


def test_special_groups():
    x = np.zeros((3, 64))
    x[1, 5] = np.inf
    x[2, 20] = np.nan
    c, b = kv4.quantise(x)
    assert np.all(c == 8) and np.all(b[0] == 0)
    assert b[1].tolist() == [0xFF, 0, 0, 0] and b[2].tolist() == [0, 0xFF, 0, 0]
    assert np.isnan(kv4.held(x)[1, :16]).all() and np.all(kv4.held(x)[1, 16:] == 0)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_page_bytes_are_each_used_once(page, d):
    """Every nibble and scale byte of a block belongs to exactly one value."""
    nib = np.zeros((kv4.block_bytes(page, d), 2), int)
    for w in range(page):
        for x in range(d):
            for at, sh in (kv4.k_code_at(w, x, page, d), kv4.v_code_at(w, x, page, d)):
                nib[at, sh // 4] += 1
        for g in range(d // 16):
            nib[kv4.k_scale_at(w, g, page, d)] += 1
            nib[kv4.v_scale_at(w, g, page, d)] += 1
    assert np.all(nib == 1)


def test_block_bytes(lib):
    for page in (16, 32, 64, 128):
        for d in (64, 128):
            assert lib.attn_kv4_block_bytes(page, d) == kv4.block_bytes(page, d)
    for page, d in ((8, 64), (48, 128), (64, 192), (256, 128), (0, 0), (-16, 64)):
        assert lib.attn_kv4_block_bytes(page, d) == 0


def test_append_and_gather_validation(lib):
    def app(k=P, v=P, cu=P, pool=P, table=P, lens=P, B=2, T=5, H=2, d=128, n=4, page=16, mp=3, ks=256, vs=256):
        return lib.attn_kv4_append(k, v, cu, pool, table, lens, B, T, H, d, n, page, mp, ks, vs, None)

    assert app(B=-1) == INVALID and app(T=-1) == INVALID and app(H=0) == INVALID and app(mp=-1) == INVALID
    assert app(d=192) == UNSUPPORTED and app(page=24) == UNSUPPORTED
    assert app(mp=1 << 28, page=128) == UNSUPPORTED     # token numbers are 32-bit
    assert app(ks=248) == INVALID                       # rows overlap
    assert app(vs=260) == MISALIGNED                    # rows are whole 16-byte units
    assert app(k=None) == INVALID and app(table=None) == INVALID and app(cu=None) == INVALID
    assert app(k=MIS) == MISALIGNED and app(pool=MIS) == MISALIGNED
    assert app(lens=ctypes.c_void_p(0x10002)) == MISALIGNED
    assert app(B=0) == OK and app(T=0) == OK            # nothing to launch

    def gat(pool=P, k=P, v=P, B=2, T=5, d=128, page=16, zero=0):
        return lib.attn_kv4_gather(pool, P, P, P, k, v, B, T, 2, d, 4, page, 3, zero, None)

    assert gat(d=96) == UNSUPPORTED and gat(page=0) == UNSUPPORTED
    assert gat(T=-3) == INVALID and gat(pool=None) == INVALID and gat(v=None) == INVALID
    assert gat(k=MIS) == MISALIGNED
    assert gat(T=0) == OK and gat(B=0) == OK


def test_decode_validation(lib):
    need = lib.attn_kv4_decode_workspace_size(2, 1, 8, 2, 128)
    assert need > 0
    assert lib.attn_kv4_decode_workspace_size(2, 1, 8, 3, 128) == 0
    assert lib.attn_kv4_decode_workspace_size(2, 1, 8, 2, 192) == 0

    def dec(q=P, pool=P, table=P, lens=P, o=P, lse=None, B=2, S=1, Hq=8, Hkv=2, d=128, page=16, window=-1, st=0,
            off=None, ws=P, wsb=need):
        return lib.attn_kv4_decode(q, pool, table, lens, o, lse, B, S, Hq, Hkv, d, 4, page, 3, ctypes.c_float(0.0),
                                   window, st, off, ws, ctypes.c_size_t(wsb), None)

    assert dec(Hq=7) == INVALID and dec(B=-1) == INVALID and dec(S=-1) == INVALID
    assert dec(d=192) == UNSUPPORTED and dec(page=20) == UNSUPPORTED
    assert dec(st=3) == INVALID and dec(st=2) == INVALID       # learnable needs the offset
    assert dec(q=None) == INVALID and dec(o=None) == INVALID and dec(lens=None) == INVALID
    assert dec(pool=None) == INVALID
    assert dec(q=MIS) == MISALIGNED and dec(lse=ctypes.c_void_p(0x10001)) == MISALIGNED
    assert dec(ws=None) == WORKSPACE and dec(wsb=need - 1) == WORKSPACE
    assert dec(ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    assert dec(B=0) == OK and dec(S=0) == OK


def test_decode_refuses_scales_past_1e30(lib):
    def dec(scale, B):
        return lib.attn_kv4_decode(P, P, P, P, P, None, B, 1, 8, 2, 128, 4, 16, 3, ctypes.c_float(scale), -1, 0, None,
                                   None, ctypes.c_size_t(0), None)

    assert dec(1.5e30, 2) == UNSUPPORTED and dec(3e38, 0) == UNSUPPORTED
    assert dec(1e30, 0) == OK and dec(float("inf"), 0) == OK and dec(-1.0, 0) == OK  # (not positive and finite: 1/sqrt(d))
    assert dec(1e30, 2) == WORKSPACE


def test_copy_pages_validation(lib):
    def cp(src, dst, n_pages=8, layers=1, byts=64, pool=P):
        a = (ctypes.c_int * max(len(src), 1))(*src)
        b = (ctypes.c_int * max(len(dst), 1))(*dst)
        return lib.attn_kv4_copy_pages(pool, layers, n_pages, ctypes.c_size_t(byts), a, b, len(src), None)

    assert cp([0, 1], [2, 2]) == INVALID       # a destination named twice
    assert cp([0, 1], [1, 2]) == INVALID       # page 1 is both
    assert cp([1, 0], [2, 1]) == INVALID
    assert cp([3], [3]) == INVALID
    assert cp([0], [8]) == INVALID and cp([-1], [2]) == INVALID and cp([9], [2]) == INVALID
    assert cp([0], [1], byts=60) == INVALID
    big = 1 << 22                              # pools past a million pages are checked by sorting
    assert cp([5, 7], [9, 9], n_pages=big) == INVALID and cp([5, 9], [9, 1], n_pages=big) == INVALID
    assert cp([5], [5], n_pages=big) == INVALID and cp([5], [big], n_pages=big) == INVALID
    assert cp([0], [1], pool=None) == INVALID and cp([0], [1], pool=MIS) == MISALIGNED
    assert cp([0], [1], n_pages=-1) == INVALID and cp([0], [1], layers=-1) == INVALID
    assert cp([0], [1], layers=70000) == UNSUPPORTED
    assert cp([], []) == OK and cp([0], [1], layers=0) == OK


def test_bad_page_status_has_a_name():
    import scaled_dot_product_tmem_gb300 as sdpa
    assert "page" in sdpa.attn_status_string(BAD_PAGE)


def test_python_refusals_without_a_gpu():
    import scaled_dot_product_tmem_gb300 as sdpa
    with pytest.raises(ValueError):
        sdpa.kv4_block_bytes(48, 128)
    pool = torch.zeros((4, 2, sdpa.kv4_block_bytes(16, 64)), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.attn_kv4_copy_pages(pool, [0], [1])
    with pytest.raises(ValueError):
        sdpa.attn_kv4_copy_pages(pool[0], [0], [1])
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.attn_kv4_append(k, k, i32(0, 3), pool, i32(0, 1).view(1, 2), i32(0))
    for bad in ([0.5], [[1]], [2 ** 40]):
        with pytest.raises(ValueError):
            sdpa._host_pages(bad, "src")
    assert sdpa._host_pages([], "src").numel() == 0
    assert sdpa._host_pages(torch.tensor([3, 4]), "src").dtype == torch.int32
