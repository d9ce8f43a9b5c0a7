"""The 4-bit paged cache on the GPU against oracle/kv4.py: appending, reading back, attention
of the newest tokens, and page copies, at ragged lengths, odd head groups, page tails and rows
that see no key.

Bounds.  Held values are exact, so append and gather are compared for equality.  Attention
rounds the probabilities and the output to bf16, each by at most 2^-8 of its value, so
  |o - o_ref| <= 2^-8 sum_j P_j |v_j| + 2^-8 |o_ref| + 2^-14 sum_j P_j |v_j|,
the last term for the fp32 arithmetic (scores to 2^-17 of sum_x |q_x k_x|, at most 30 or so in
these cases, exponentials and sums to 2^-20).  A score is an fp32 sum of d <= 128 products:
off by at most d 2^-24 = 2^-17 of scale sum_x |q_x k_jx|; the exponential, sum and logarithm
add 2^-18 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu


def _sdpa():
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _clean():
    torch.cuda.synchronize()
    st, site = _sdpa().attn_last_device_error()
    assert st == 0, f"device error status {st} site {site:#x}"


def _cu(lens):
    return _i32([0] + np.cumsum(lens).tolist())


def _table(gen, need, extra=2):
    """Pages in random order; unused entries are -1."""
    n_pages = sum(need) + extra
    perm = torch.randperm(n_pages, generator=gen).tolist()
    t = torch.full((len(need), max(max(need, default=0), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    return t, n_pages


class Cache:
    """A filled cache with the fp64 values its tokens are held as.  The pool starts as 0xFF
    bytes: unwritten places have NaN scales."""

    def __init__(self, lens, H_kv, d, page, seed=0, big=1.0):
        sdpa = _sdpa()
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.d = lens, page, d
        T = sum(lens)
        k = (torch.randn((T, H_kv, d), generator=gen) * big).to(torch.bfloat16)
        v = torch.randn((T, H_kv, d), generator=gen).to(torch.bfloat16)
        table, n_pages = _table(gen, [-(-n // page) for n in lens])
        self.table = table.cuda()
        self.pool = sdpa.kv4_pool(n_pages, H_kv, d, page).fill_(0xFF)
        self.seq_lens = _i32(lens)
        self.k, self.v = kv4.held(k.double().numpy()), kv4.held(v.double().numpy())
        self.kt, self.vt = k, v
        self.at = np.cumsum([0] + list(lens))
        sdpa.attn_kv4_append(k.cuda(), v.cuda(), _cu(lens), self.pool, self.table, _i32([0] * len(lens)))


def _check_decode(c, q, o, lse, **kw):
    q, o = q.double().cpu().numpy(), o.double().cpu().numpy()
    for b, L in enumerate(c.lens):
        sl = slice(int(c.at[b]), int(c.at[b + 1]))
        ro, rl, a, mag = kv4.decode(q[b], c.k[sl], c.v[sl], L, **kw)
        bound = 2.0 ** -8 * (a + np.abs(ro)) + 2.0 ** -14 * a
        err = np.abs(o[b] - ro)
        assert np.all(err <= bound), f"entry {b} (len {L}): o off by {np.max(err - bound)} more than its bound"
        if lse is not None:
            g = lse[b].double().cpu().numpy()
            fin = np.isfinite(rl)
            assert np.array_equal(g[~fin], rl[~fin]), f"entry {b}: lse of rows without a key"
            tol = 2.0 ** -17 * mag + 2.0 ** -18 * (1 + np.abs(np.where(fin, rl, 0)))
            assert np.all(np.abs(g - rl)[fin] <= tol[fin]), f"entry {b}: lse off by {np.max(np.abs(g - rl)[fin])}"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_bytes_and_gather(page, d):
    """The pool's bytes are the format's, in two appends of ragged rows; bytes of no token stay;
    reading back gives the held values, and rows past the last sequence are left alone."""
    sdpa = _sdpa()
    gen = torch.Generator().manual_seed(page + d)
    H, first, second = 3, [5, 0, 33, 1], [1, 17, 0, 2 * page]
    need = [-(-(a + b) // page) for a, b in zip(first, second)]
    table, n_pages = _table(gen, need)
    pool = torch.full((n_pages, H, sdpa.kv4_block_bytes(page, d)), 0xA5, dtype=torch.uint8, device="cuda")
    ref = pool.cpu().numpy().copy()
    start = [0] * 4
    tok = [[], [], [], []]
    for lens in (first, second):
        T = sum(lens)
        rows = T + 3  # three rows of no sequence
        x = torch.randn((2, rows, H, d), generator=gen) * 10.0 ** torch.empty(2, rows, H, 1).uniform_(-6, 3, generator=gen)
        k, v = x[0].to(torch.bfloat16), x[1].to(torch.bfloat16)
        sdpa.attn_kv4_append(k.cuda(), v.cuda(), _cu(lens), pool, table.cuda(), _i32(start))
        at = 0
        for b, n in enumerate(lens):
            for i in range(n):
                pos = start[b] + i
                for h in range(H):
                    kv4.write_token(ref[table[b, pos // page], h], pos % page, k[at, h].double().numpy(),
                                    v[at, h].double().numpy(), page)
                tok[b].append((k[at], v[at]))
                at += 1
            start[b] += n
    _clean()
    assert np.array_equal(pool.cpu().numpy(), ref)
    total = sum(start)
    ko = torch.full((total + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    sdpa.attn_kv4_gather(pool, table.cuda(), _cu(start), _i32([0] * 4), ko, vo)
    _clean()
    k = torch.stack([t[0] for b in tok for t in b]).double().numpy()
    v = torch.stack([t[1] for b in tok for t in b]).double().numpy()
    assert np.array_equal(ko[:total].double().cpu().numpy(), kv4.held(k))
    assert np.array_equal(vo[:total].double().cpu().numpy(), kv4.held(v))
    assert torch.all(ko[total:] == 7) and torch.all(vo[total:] == 7)
    # from the middle of the sequences, into new tensors with zeroed spare rows
    k2, v2 = sdpa.kv4_gather(pool, table.cuda(), _cu([2, 1, 0, 4]), _i32([3, 16, 0, page - 1]), 9, d)
    _clean()
    off = np.cumsum([0] + start)
    pick = [off[0] + 3, off[0] + 4, off[1] + 16] + [off[3] + page - 1 + i for i in range(4)]
    assert np.array_equal(k2[:7].double().cpu().numpy(), kv4.held(k)[pick])
    assert np.array_equal(v2[:7].double().cpu().numpy(), kv4.held(v)[pick])
    assert torch.all(k2[7:] == 0) and torch.all(v2[7:] == 0)


def test_append_from_slices_of_a_fused_projection():
    sdpa = _sdpa()
    H, d, page, T = 2, 64, 16, 21
    qkv = torch.randn((T, 8 * d + 2 * H * d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    k = qkv[:, 8 * d:8 * d + H * d].view(T, H, d)
    v = qkv[:, 8 * d + H * d:].view(T, H, d)
    table = _i32([[1, 0]])
    a, b = (sdpa.kv4_pool(2, H, d, page).zero_() for _ in range(2))
    sdpa.attn_kv4_append(k, v, _i32([0, T]), a, table, _i32([0]))
    sdpa.attn_kv4_append(k.contiguous(), v.contiguous(), _i32([0, T]), b, table, _i32([0]))
    _clean()
    assert torch.equal(a, b)
    with pytest.raises(ValueError):
        sdpa.attn_kv4_append(k.transpose(1, 2), v, _i32([0, T]), a, table, _i32([0]))


def test_special_values_are_held_as_nan_and_extremes_saturate():
    sdpa = _sdpa()
    H, d, page = 1, 64, 16
    x = torch.zeros((6, H, d), dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 17], x[2, 0, 40] = float("inf"), float("nan"), -float("inf")
    x[3, 0, :] = 3e38                              # past 7 x 61440
    x[4, 0, ::2], x[4, 0, 1::2] = 1e-40, -2e-6     # subnormal numbers, and scales below 2^-14
    x[5, 0, :16] = torch.linspace(-3, 3, 16)
    pool, table = sdpa.kv4_pool(1, H, d, page), _i32([[0]])
    sdpa.attn_kv4_append(x.cuda(), x.cuda(), _i32([0, 6]), pool, table, _i32([0]))
    k, v = sdpa.kv4_gather(pool, table, _i32([0, 6]), _i32([0]), 6, d)
    _clean()
    ref = kv4.held(x.double().numpy())
    for got in (k, v):
        assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)
    assert ref[3].max() == 7 * 61440


# name, lens, S_q, H_q, H_kv, d, page, window, sink
DECODE = [
    ("gqa4_d128_ragged", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 300], 1, 8, 2, 128, 64, -1, "vanilla"),
    ("gqa4_d64_page16", [200, 1, 16, 15, 97], 1, 8, 2, 64, 16, -1, "vanilla"),
    ("empty_entries", [0, 5, 0, 70], 1, 4, 2, 128, 32, -1, "off_by_one"),
    ("more_queries_than_tokens", [2, 0, 1, 9], 4, 4, 2, 64, 16, -1, "vanilla"),
    ("mha", [77, 130], 1, 4, 4, 128, 128, -1, "learnable"),
    ("mqa32", [600, 33], 1, 32, 1, 128, 64, -1, "vanilla"),
    ("mqa32_two_tokens", [257, 64], 2, 32, 1, 64, 32, -1, "learnable"),
    ("group7_odd", [90, 41], 1, 7, 1, 128, 16, -1, "off_by_one"),
    ("group6_three_tokens", [50, 129, 3], 3, 24, 4, 128, 64, -1, "vanilla"),
    ("window", [500, 20, 130, 1], 1, 8, 2, 128, 64, 100, "vanilla"),
    ("window0_only_itself", [40, 1], 2, 4, 2, 64, 16, 0, "vanilla"),
    ("window_multi_token_sink", [300, 65], 5, 4, 2, 64, 128, 33, "learnable"),
    ("huge_window_short_entries", [2, 40, 0], 4, 4, 2, 64, 16, 2 ** 31 - 1, "vanilla"),
    ("window_past_32_bits", [200], 1, 4, 2, 64, 16, 2 ** 40, "vanilla"),
    ("long_context", [5000, 1, 2600], 1, 8, 2, 128, 64, -1, "vanilla"),
    ("long_prompt_of_queries", [150], 100, 4, 2, 64, 32, -1, "vanilla"),
]


@pytest.mark.parametrize("case", DECODE, ids=[c[0] for c in DECODE])
def test_decode(case):
    _, lens, S_q, H_q, H_kv, d, page, window, sink = case
    sdpa = _sdpa()
    c = Cache(lens, H_kv, d, page, seed=len(lens))
    gen = torch.Generator().manual_seed(99)
    q = torch.randn((len(lens), S_q, H_q, d), generator=gen).to(torch.bfloat16)
    off = torch.randn(H_q, generator=gen)
    ref_sink = {"vanilla": None, "off_by_one": np.zeros(H_q), "learnable": off.double().numpy()}[sink]
    kw = dict(window=window, softmax_type=sink, softmax_offset=off.cuda() if sink == "learnable" else None)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, **kw)
    o2, lse2 = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, **kw)
    _clean()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # bitwise reproducible
    _check_decode(c, q, o, lse, window=window, sink=ref_sink)


def test_decode_scale_large_scores_and_no_lse():
    """Scores far apart (the running maximum moves often) and a scale of the caller's."""
    sdpa = _sdpa()
    c = Cache([700, 129], 2, 128, 64, seed=5, big=20.0)
    q = torch.randn((2, 1, 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    o = torch.empty((2, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    sdpa.attn_kv4_decode(q.cuda(), c.pool, c.table, c.seq_lens, o, scale=0.01)
    _clean()
    _check_decode(c, q, o, None, scale=0.01)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens)
    _clean()
    # scores of magnitude 500 and more: the scores' own fp32 error (2^-17 sum |q k|) reaches o
    rq = q.double().numpy()
    for b in range(2):
        sl = slice(int(c.at[b]), int(c.at[b + 1]))
        ro, rl, a, mag = kv4.decode(rq[b], c.k[sl], c.v[sl], c.lens[b])
        slack = np.expm1(2 * 2.0 ** -17 * mag.T)[..., None]
        err = np.abs(o[b].double().cpu().numpy() - ro)
        assert np.all(err <= (2.0 ** -8 + 2.0 ** -14 + slack) * a + 2.0 ** -8 * np.abs(ro))
        assert np.all(np.abs(lse[b].double().cpu().numpy() - rl) <= 2.0 ** -17 * mag + 2.0 ** -18 * (1 + np.abs(rl)))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_over_the_whole_range_of_scales(d):
    """Groups of 16 dims with scales from a few 2^-17 to tens of thousands side by side."""
    sdpa = _sdpa()
    gen, L, page = torch.Generator().manual_seed(8), 150, 32
    k = torch.randn((L, 1, d), generator=gen)
    k[..., :32] *= 2.0 ** -14
    v = torch.randn((L, 1, d), generator=gen) * torch.logspace(-14, 16, d // 16, base=2.0).repeat_interleave(16)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c = Cache([L], 1, d, page)
    sdpa.attn_kv4_append(k.cuda(), v.cuda(), _cu([L]), c.pool, c.table, _i32([0]))
    c.k, c.v = kv4.held(k.double().numpy()), kv4.held(v.double().numpy())
    assert 0 < np.abs(c.v[..., :16]).max() < 2.0 ** -11 and np.abs(c.v[..., -16:]).max() >= 2.0 ** 17
    assert np.abs(c.k[..., :32]).max() > 0
    q = torch.randn((1, 1, 4, d), generator=gen).to(torch.bfloat16)
    q[..., :32] *= 2.0 ** 14
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens)
    _clean()
    _check_decode(c, q, o, lse)


def test_decode_window_and_queries_past_32_bits_together():
    """A table of 2^31 - 128 tokens, a window of nearly all of them and more queries than tokens:
    the window's first key lies below -2^31."""
    sdpa = _sdpa()
    c = Cache([1, 130], 1, 64, 128)
    table = torch.full((2, 2 ** 24 - 1), -1, dtype=torch.int32, device="cuda")
    table[:, :2] = c.table
    q = torch.randn((2, 200, 4, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, table, c.seq_lens, window=2 ** 31 - 130)
    _clean()
    _check_decode(c, q, o, lse)


def test_decode_nan_reaches_its_own_head_and_entry_only():
    sdpa = _sdpa()
    c = Cache([40, 40], 2, 64, 16, seed=8)
    bad = c.vt[:1].clone()
    bad[0, 0, 3] = float("nan")
    sdpa.attn_kv4_append(c.kt[7:8].cuda(), bad.cuda(), _i32([0, 1, 1]), c.pool, c.table, _i32([7, 0]))
    q = torch.randn((2, 1, 4, 64), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    o, lse = sdpa.sdpa_decode_kv4(q, c.pool, c.table, c.seq_lens)
    _clean()
    assert torch.isnan(o[0, 0, :2, :16]).all() and torch.isfinite(o[0, 0, :2, 16:]).all()
    assert torch.isfinite(o[0, 0, 2:]).all() and torch.isfinite(o[1]).all() and torch.isfinite(lse).all()
    # outside the window the token is not seen
    o, lse = sdpa.sdpa_decode_kv4(q, c.pool, c.table, c.seq_lens, window=20)
    _clean()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_pages_outside_the_pool_read_as_zeros_and_are_reported():
    sdpa = _sdpa()
    c = Cache([40, 20], 2, 64, 16, seed=10)
    table = c.table.clone()
    table[0, 1], table[1, 0] = -7, c.pool.shape[0] + 5
    q = torch.randn((2, 1, 4, 64), generator=torch.Generator().manual_seed(11)).to(torch.bfloat16)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, table, c.seq_lens)
    torch.cuda.synchronize()
    assert sdpa.attn_last_device_error() == (7, 3)
    assert sdpa.attn_last_device_error()[0] == 0
    c.k[16:32], c.v[16:32], c.k[40:56], c.v[40:56] = 0, 0, 0, 0
    _check_decode(c, q, o, lse)
    k, v = sdpa.kv4_gather(c.pool, table, _cu(c.lens), _i32([0, 0]), 60, 64)
    torch.cuda.synchronize()
    assert sdpa.attn_last_device_error() == (7, 2)
    assert np.array_equal(k.double().cpu().numpy(), c.k) and np.array_equal(v.double().cpu().numpy(), c.v)
    before = c.pool.clone()
    one = c.kt[:2].cuda()
    sdpa.attn_kv4_append(one, one, _i32([0, 1, 2]), c.pool, table, _i32([20, 4000]))  # a bad page; past the table
    torch.cuda.synchronize()
    assert sdpa.attn_last_device_error() == (7, 1)
    assert torch.equal(before, c.pool)


def test_lengths_past_the_table_are_clamped():
    sdpa = _sdpa()
    c = Cache([32, 32], 2, 64, 16, seed=12)
    q = torch.randn((2, 1, 4, 64), generator=torch.Generator().manual_seed(13)).to(torch.bfloat16)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, _i32([1000, -4]))
    _clean()
    c.lens = [32, 0]
    c.at = np.array([0, 32, 32])
    _check_decode(c, q, o, lse)


def test_copy_pages():
    sdpa = _sdpa()
    gen = torch.Generator().manual_seed(14)
    for shape in ((40, 3, sdpa.kv4_block_bytes(16, 64)), (2, 1200, 1, sdpa.kv4_block_bytes(32, 128)),
                  (9500, 1, sdpa.kv4_block_bytes(16, 64))):  # more pairs than one launch takes
        pool = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
        n_pages = shape[-3]
        perm = torch.randperm(n_pages, generator=gen)
        n = n_pages // 2 - 1
        src, dst = perm[:n].clone(), perm[n:2 * n]
        src[1::3] = src[0]  # one source, many destinations
        ref = pool.clone()
        ref[..., dst, :, :] = pool[..., src, :, :]
        got = pool.cuda()
        sdpa.attn_kv4_copy_pages(got, src, dst.to(torch.int32))
        _clean()
        assert torch.equal(got.cpu(), ref)
        with pytest.raises(sdpa.AttnError, match="invalid"):
            sdpa.attn_kv4_copy_pages(got, [0, 1], [1, 2])
        assert torch.equal(got.cpu(), ref)
    sdpa.attn_kv4_copy_pages(got, [], [])


def test_pages_past_4_gb():
    """Pages whose bytes lie past 2^32: append, gather, decode and copy address them."""
    sdpa = _sdpa()
    H, d, page, n_pages = 8, 128, 64, 62000  # 73,728 bytes a page: 4.57 GB
    pool = sdpa.kv4_pool(n_pages, H, d, page)
    lens = [130, 70]
    gen = torch.Generator().manual_seed(15)
    k, v = (torch.randn((200, H, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    table = _i32([[61999, 3, 60000], [59999, 61000, -1]])
    sdpa.attn_kv4_append(k.cuda(), v.cuda(), _cu(lens), pool, table, _i32([0, 0]))
    kk, vv = sdpa.kv4_gather(pool, table, _cu(lens), _i32([0, 0]), 200, d)
    q = torch.randn((2, 1, 16, d), generator=gen).to(torch.bfloat16)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), pool, table, _i32(lens))
    sdpa.attn_kv4_copy_pages(pool, [61999, 60000, 59999], [5, 61500, 61998])
    moved = _i32([[5, 3, 61500], [61998, 61000, -1]])
    o2, lse2 = sdpa.sdpa_decode_kv4(q.cuda(), pool, moved, _i32(lens))
    _clean()
    c = Cache.__new__(Cache)
    c.lens, c.at = lens, np.array([0, 130, 200])
    c.k, c.v = kv4.held(k.double().numpy()), kv4.held(v.double().numpy())
    assert np.array_equal(kk.double().cpu().numpy(), c.k) and np.array_equal(vv.double().cpu().numpy(), c.v)
    _check_decode(c, q, o, lse)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_refusals():
    sdpa = _sdpa()
    c = Cache([20], 2, 64, 16)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    bad = [
        (q.half(), c.pool, c.table, c.seq_lens), (q[:, :, ::2], c.pool, c.table, c.seq_lens),
        (q, c.pool[:, :, :-16].contiguous(), c.table, c.seq_lens), (q, c.pool, c.table.long(), c.seq_lens),
        (q, c.pool, c.table, _i32([1, 2])), (q.expand(2, 1, 4, 64).contiguous(), c.pool, c.table, c.seq_lens),
        (q, c.pool.cpu(), c.table, c.seq_lens),
    ]
    for args in bad:
        with pytest.raises((TypeError, ValueError)):
            sdpa.sdpa_decode_kv4(*args)
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_decode_kv4(q, c.pool, c.table, c.seq_lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_decode_kv4(q[:, :, :3].contiguous(), c.pool, c.table, c.seq_lens)
    with pytest.raises(ValueError):
        sdpa.sdpa_decode_kv4(q, c.pool, c.table, c.seq_lens, softmax_type="learnable",
                             softmax_offset=torch.zeros(3, device="cuda"))


def test_calls_on_two_streams_at_once():
    """Decodes and appends of two caches, many times over on two streams without waiting for each
    other, give the bits of the same calls one at a time."""
    sdpa = _sdpa()
    caches = [Cache([900, 33, 2000], 2, 128, 64, seed=30), Cache([70, 1500, 5, 641], 2, 64, 16, seed=31)]
    gen = torch.Generator().manual_seed(32)
    qs = [torch.randn((len(c.lens), 1, 8, c.d), generator=gen).to(torch.bfloat16).cuda() for c in caches]
    alone = [sdpa.sdpa_decode_kv4(q, c.pool, c.table, c.seq_lens) for q, c in zip(qs, caches)]
    news = [(c.kt[:len(c.lens)].cuda(), c.vt[:len(c.lens)].cuda(), _cu([1] * len(c.lens)), c.seq_lens - 1) for c in caches]
    _clean()
    streams = [torch.cuda.Stream() for _ in caches]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(caches, streams)):
            with torch.cuda.stream(s):
                out[i].append(sdpa.sdpa_decode_kv4(qs[i], c.pool, c.table, c.seq_lens))
    for i, (c, s) in enumerate(zip(caches, streams)):  # and with new last tokens
        k, v, cu, start = news[i]
        sdpa.attn_kv4_append(k, v, cu, c.pool, c.table, start, stream=s)
        out[i].append(sdpa.sdpa_decode_kv4(qs[i], c.pool, c.table, c.seq_lens, stream=s))
    for s in streams:
        s.synchronize()
    _clean()
    for i, c in enumerate(caches):
        for o, lse in out[i][:-1]:
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1])
        for b, end in enumerate(c.at[1:]):
            c.k[end - 1], c.v[end - 1] = (kv4.held(t[b].double().cpu().numpy()) for t in news[i][:2])
        _check_decode(c, qs[i], *out[i][-1])


def test_serving_loop_captured_and_on_another_stream():
    """Prompts enter the cache, a request forks, and each step appends one token and attends: the
    steps run eagerly on a side stream and again as a captured graph, with the same bits."""
    sdpa = _sdpa()
    H_q, H_kv, d, page, steps = 8, 2, 128, 16, 20
    gen = torch.Generator().manual_seed(21)
    lens = [37, 5, 37]  # the third request is a fork of the first
    prompt = [torch.randn((42, H_kv, d), generator=gen).to(torch.bfloat16) for _ in range(2)]
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0], table[1, :2], table[2] = torch.tensor([5, 0, 3, 7]), torch.tensor([2, 6]), torch.tensor([5, 0, 9, 8])
    new = [torch.randn((steps, 3, H_kv, d), generator=gen).to(torch.bfloat16) for _ in range(2)]
    qs = torch.randn((steps, 3, 1, H_q, d), generator=gen).to(torch.bfloat16).cuda()

    def fill():
        pool = sdpa.kv4_pool(10, H_kv, d, page).fill_(0xFF)
        sdpa.attn_kv4_append(prompt[0].cuda(), prompt[1].cuda(), _cu([37, 5, 0]), pool, table.cuda(), _i32([0, 0, 0]))
        sdpa.attn_kv4_copy_pages(pool, [3], [9])  # the fork's own copy of the partly filled page
        return pool

    k1, v1 = (t.cuda() for t in new)
    cu, one = _cu([1, 1, 1]), _i32([1, 1, 1])
    tab = table.cuda()
    # eager, on a side stream
    side = torch.cuda.Stream()
    pool, n = fill(), _i32(lens)
    side.wait_stream(torch.cuda.current_stream())
    eager = []
    with torch.cuda.stream(side):
        for i in range(steps):
            sdpa.attn_kv4_append(k1[i], v1[i], cu, pool, tab, n)
            n.add_(one)
            eager.append(sdpa.sdpa_decode_kv4(qs[i], pool, tab, n))
    side.synchronize()
    _clean()
    # one captured step, replayed
    pool2, n2 = fill(), _i32(lens)
    kk, vv, qq = k1[0].clone(), v1[0].clone(), qs[0].clone()
    ws = torch.empty(max(256, sdpa.attn_kv4_decode_workspace_size(3, 1, H_q, H_kv, d)), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(qq), torch.empty((3, H_q, 1), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdpa.attn_kv4_append(kk, vv, cu, pool2, tab, n2)
        n2.add_(one)
        sdpa.attn_kv4_decode(qq, pool2, tab, n2, o, lse, workspace=ws)
    for i in range(steps):
        kk.copy_(k1[i]), vv.copy_(v1[i]), qq.copy_(qs[i])
        g.replay()
        assert torch.equal(o, eager[i][0]) and torch.equal(lse, eager[i][1]), f"step {i}"
    _clean()
    assert torch.equal(pool, pool2)
    # the last step against the oracle: each request's own tokens
    c = Cache.__new__(Cache)
    c.lens = [n + steps for n in lens]
    toks = [[(t[:37], t[37:42], t[:37])[b] for b in range(3)] for t in prompt]
    k, v = (np.concatenate([torch.cat([toks[w][b], new[w][:, b]]).double().numpy() for b in range(3)]) for w in (0, 1))
    c.k, c.v, c.at = kv4.held(k), kv4.held(v), np.cumsum([0] + c.lens)
    _check_decode(c, qs[-1], eager[-1][0], eager[-1][1])


def _spoil(c, places):
    """The value of token `pos` of entry b, head h, gets a NaN in dim x: for (b, pos, h, x) in places."""
    sdpa = _sdpa()
    for b, pos, h, x in places:
        at = int(c.at[b]) + pos
        c.vt[at, h, x] = float("nan")
        one = [int(i == b) for i in range(len(c.lens))]
        start = [pos if i == b else 0 for i in range(len(c.lens))]
        sdpa.attn_kv4_append(c.kt[at:at + 1].cuda(), c.vt[at:at + 1].cuda(), _cu(one), c.pool, c.table, _i32(start))
        c.v[at] = kv4.held(c.vt[at].double().numpy())


def _check_decode_with_nans(c, q, o, lse, **kw):
    """o is NaN where the oracle's is, and there only; the rest within the bounds of _check_decode."""
    q, o, lse = q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy()
    count = 0
    for b, L in enumerate(c.lens):
        sl = slice(int(c.at[b]), int(c.at[b + 1]))
        ro, rl, a, mag = kv4.decode(q[b], c.k[sl], c.v[sl], L, **kw)
        nan = np.isnan(ro)
        count += nan.sum()
        assert np.array_equal(np.isnan(o[b]), nan), f"entry {b} (len {L}): NaN in other places"
        bound = np.where(nan, 0, 2.0 ** -8 * (a + np.abs(ro)) + 2.0 ** -14 * a)
        assert np.all(np.where(nan, 0, np.abs(o[b] - ro)) <= bound), f"entry {b} (len {L})"
        fin = np.isfinite(rl)
        assert np.array_equal(lse[b][~fin], rl[~fin])
        tol = 2.0 ** -17 * mag + 2.0 ** -18 * (1 + np.abs(np.where(fin, rl, 0)))
        assert np.all(np.abs(np.where(fin, lse[b], 0) - np.where(fin, rl, 0)) <= tol)
    return count


# name, lens, S_q, H_q, H_kv, d, page, window, tokens from the end that hold a NaN
NAN_HIDDEN = [
    ("newest_of_two", [40, 33, 128, 129], 2, 4, 2, 64, 16, -1, [1]),
    ("newest_of_two_d128", [40, 33, 128, 129], 2, 8, 2, 128, 64, -1, [1]),
    ("middle_of_four", [70, 4, 257], 4, 4, 2, 128, 32, -1, [2]),
    ("window_leaves_it", [200, 61, 300], 3, 4, 2, 128, 64, 20, [23, 21]),
    ("window_leaves_it_d64", [200, 61, 300], 3, 8, 1, 64, 16, 40, [43, 42]),
    ("both_ends", [160, 500], 5, 6, 2, 64, 128, 33, [37, 1]),
    ("rows_16", [90, 300], 4, 4, 1, 128, 16, -1, [1, 2]),
    ("rows_32_window", [90, 300, 33], 4, 16, 2, 128, 64, 64, [1, 67]),
    ("rows_past_32", [150, 70], 50, 4, 2, 64, 32, -1, [1, 25, 49]),
    ("rows_past_32_window", [400], 70, 8, 2, 128, 64, 100, [1, 65, 130]),
    ("seen_by_all", [90, 65], 2, 4, 2, 64, 16, -1, [2, 30]),
    ("long", [6000, 1], 3, 4, 1, 128, 64, 4000, [1, 2, 4003, 3000]),
    ("more_queries_than_tokens", [2, 1, 9], 4, 4, 2, 64, 16, -1, [1]),
]


@pytest.mark.parametrize("case", NAN_HIDDEN, ids=[c[0] for c in NAN_HIDDEN])
def test_decode_nan_reaches_only_queries_that_see_its_token(case):
    """A token held as NaN reaches the queries that see it, in its own 16 dims and kv head, and no other
    query: not those before a proposed token, nor those whose window it has left."""
    name, lens, S_q, H_q, H_kv, d, page, window, back = case
    c = Cache(lens, H_kv, d, page, seed=len(name))
    places = [(b, L - n, (b + n) % H_kv, (37 * n + b) % d) for b, L in enumerate(lens) for n in back if n <= L]
    _spoil(c, places)
    q = torch.randn((len(lens), S_q, H_q, d), generator=torch.Generator().manual_seed(51)).to(torch.bfloat16)
    sdpa = _sdpa()
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, window=window, softmax_type="off_by_one")
    o2, lse2 = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, window=window, softmax_type="off_by_one")
    _clean()
    assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(o2)) and torch.equal(lse, lse2)
    n = _check_decode_with_nans(c, q, o, lse, window=window, sink=np.zeros(H_q))
    assert n > 0 and n < o.numel()


def test_decode_nan_of_a_token_without_weight_is_kept():
    """A sequence whose first tokens outweigh all others by more than fp32 holds: a NaN value that a
    query sees reaches it from any place in the sequence, however little its token weighs."""
    sdpa = _sdpa()
    L, H, d, page = 6000, 4, 128, 64
    c = Cache([L], 1, d, page, seed=61)
    q = torch.randn((1, 1, H, d), generator=torch.Generator().manual_seed(62)).to(torch.bfloat16)
    # keys along the sum of the queries: scores of the first tokens above the others' by hundreds
    c.kt[:64] = (q[0, 0].float().sum(0) * 20).to(torch.bfloat16)
    sdpa.attn_kv4_append(c.kt.cuda(), c.vt.cuda(), _i32([0, L]), c.pool, c.table, _i32([0]))
    s = q[0, 0].double().numpy() @ kv4.held(c.kt.double().numpy())[:, 0].T / np.sqrt(d)
    assert (s[:, :64].min(1) - s[:, 64:].max(1)).min() > 128  # exp2(-128 log2(e)) is 0 in fp32
    bad = c.vt[:1].clone()
    bad[0, 0, 20] = float("nan")
    outs = []
    for at in range(64, L, 101):
        sdpa.attn_kv4_append(c.kt[at:at + 1].cuda(), bad.cuda(), _i32([0, 1]), c.pool, c.table, _i32([at]))
        outs.append((at, *sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens)))
        sdpa.attn_kv4_append(c.kt[at:at + 1].cuda(), c.vt[at:at + 1].cuda(), _i32([0, 1]), c.pool, c.table, _i32([at]))
    _clean()
    for at, o, lse in outs:
        assert torch.isnan(o[0, 0, :, 16:32]).all(), f"token {at}"
        assert torch.isfinite(o[0, 0, :, :16]).all() and torch.isfinite(o[0, 0, :, 32:]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("window,S_q", [(0, 1), (1, 2), (15, 1), (40, 3), (127, 1), (200, 40)])
def test_decode_needs_no_page_before_the_window(page, d, window, S_q):
    """Pages whose tokens every query's window has left may be gone from the table (a negative entry, or one
    outside the pool): nothing is reported, and the outputs are those of the whole cache."""
    sdpa = _sdpa()
    lens = [1, 127, 128, 129, 255, 256, 270, 333, 600, 641, 0, 1000]
    c = Cache(lens, 2, d, page, seed=window)
    q = torch.randn((len(lens), S_q, 4, d), generator=torch.Generator().manual_seed(71)).to(torch.bfloat16)
    whole = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, window=window)
    table, gone = c.table.clone(), 0
    for b, L in enumerate(lens):
        n = max(0, L - S_q - window) // page  # pages whose last token lies before the first query's window
        table[b, :n] = torch.tensor([(-1, c.pool.shape[0], -2 ** 31, 2 ** 31 - 1)[i % 4] for i in range(n)], dtype=torch.int32)
        gone += n
    assert gone > 0
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, table, c.seq_lens, window=window)
    _clean()
    assert torch.equal(o, whole[0]) and torch.equal(lse, whole[1])
    _check_decode(c, q, o, lse, window=window)
    # the first page that the window reaches is still needed
    b = lens.index(1000)
    table[b, max(0, 1000 - S_q - window) // page] = -1
    sdpa.sdpa_decode_kv4(q.cuda(), c.pool, table, c.seq_lens, window=window)
    torch.cuda.synchronize()
    assert sdpa.attn_last_device_error() == (7, 3)


# sequences: up to 32 fit one lane each, beyond that they are taken in groups of 32
@pytest.mark.parametrize("B", [31, 32, 33, 64, 65, 97, 200])
@pytest.mark.parametrize("window,S_q,sink", [(-1, 1, "vanilla"), (60, 3, "learnable")])
def test_decode_of_many_sequences(B, window, S_q, sink):
    """Empty sequences across a border between groups, a long one that spans several blocks in the
    middle, the rest of any short length."""
    sdpa = _sdpa()
    H_q, H_kv, d, page = 4, 2, 64, 32
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 200, B)
    lens[28:35] = 0
    if B > 64:
        lens[60:66] = 0
    lens[B // 2] = 5000
    lens[-1] = 77
    lens = lens.tolist()
    c = Cache(lens, H_kv, d, page, seed=B)
    gen = torch.Generator().manual_seed(81)
    q = torch.randn((B, S_q, H_q, d), generator=gen).to(torch.bfloat16)
    off = torch.randn(H_q, generator=gen)
    kw = dict(window=window, softmax_type=sink, softmax_offset=off.cuda() if sink == "learnable" else None)
    o, lse = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, **kw)
    o2, lse2 = sdpa.sdpa_decode_kv4(q.cuda(), c.pool, c.table, c.seq_lens, **kw)
    _clean()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_decode(c, q, o, lse, window=window, sink=off.double().numpy() if sink == "learnable" else None)


@pytest.mark.parametrize("B", [16, 17, 18, 256, 257, 258, 1000, 4100])
def test_append_and_gather_of_many_sequences(B):
    """The search for a row's sequence takes 16 ways a step: one more step past 16, 256 and 4096
    sequences.  Runs of empty sequences, and rows of no sequence behind the last."""
    sdpa = _sdpa()
    H, d, page = 1, 64, 16
    rng = np.random.default_rng(B)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(0, 4, B))
    new[B // 3:B // 3 + 40] = 0
    new[-1] = 2
    start = rng.integers(0, 30, B)
    T = int(new.sum())
    gen = torch.Generator().manual_seed(B)
    table, n_pages = _table(gen, [-(-int(a + b) // page) for a, b in zip(start, new)])
    k, v = (torch.randn((T + 5, H, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    pool = torch.full((n_pages, H, sdpa.kv4_block_bytes(page, d)), 0xA5, dtype=torch.uint8, device="cuda")
    ref = pool.cpu().numpy().copy()
    cu, st = _cu(new.tolist()), _i32(start.tolist())
    sdpa.attn_kv4_append(k.cuda(), v.cuda(), cu, pool, table.cuda(), st)
    t = 0
    for b in range(B):
        for i in range(int(new[b])):
            pos = int(start[b]) + i
            kv4.write_token(ref[table[b, pos // page], 0], pos % page, k[t, 0].double().numpy(), v[t, 0].double().numpy(), page)
            t += 1
    _clean()
    assert np.array_equal(pool.cpu().numpy(), ref)
    ko, vo = sdpa.kv4_gather(pool, table.cuda(), cu, st, T + 5, d)
    _clean()
    assert np.array_equal(ko[:T].double().cpu().numpy(), kv4.held(k[:T].double().numpy()))
    assert np.array_equal(vo[:T].double().cpu().numpy(), kv4.held(v[:T].double().numpy()))
    assert torch.all(ko[T:] == 0) and torch.all(vo[T:] == 0)
