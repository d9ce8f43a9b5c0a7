"""Drafted trees over the 4-bit cache on the GPU against oracle/tree.py: ragged trees and prefixes, chains,
windows, sinks, page tails, NaN tokens beside the path, missing pages, and the accepted nodes' moves.

Bounds.  Held values are exact.  The probabilities and the output are rounded to bf16, each by at most
2^-8 of its value, so
  |o - o_ref| <= 2^-8 sum_j P_j |v_j| + 2^-8 |o_ref| + 2^-14 sum_j P_j |v_j|,
the last term for the fp32 arithmetic (scores to 2^-17 of sum_x |q_x k_x|, at most 30 or so in these
cases, exponentials and sums to 2^-20).  A score is an fp32 sum of d <= 128 products: off by at most d 2^-24
= 2^-17 of scale sum_x |q_x k_jx|; the exponential, sum and logarithm add 2^-18 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from oracle import kv4, tree

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


def _parents(rng, nodes):
    return [int(rng.integers(max(-1, i - 5), i)) for n in nodes for i in range(n)]


class Trees:
    """Sequences of L tokens before a tree of n nodes each, all in the cache; the pool starts as 0xFF bytes, so
    that unwritten places have NaN scales."""

    def __init__(self, lens, nodes, H, H_kv, d, page, seed=0, chain=False, extra_rows=0, edit=None):
        sdpa = _sdpa()
        rng = np.random.default_rng(seed)
        self.lens, self.nodes, self.page, self.d, self.H = lens, nodes, page, d, H
        total = [L + n for L, n in zip(lens, nodes)]
        need = [-(-t // page) for t in total]
        perm = rng.permutation(sum(need) + 2)
        tab = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            tab[b, :m] = perm[at:at + m]
            at += m
        self.table = _i32(tab.tolist())
        self.pool = sdpa.kv4_pool(sum(need) + 2, H_kv, d, page).fill_(0xFF)
        gen = torch.Generator().manual_seed(seed)
        T = sum(total)
        k, v = (torch.randn((T, H_kv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
        self.at = np.cumsum([0] + total)
        if edit is not None:
            edit(self, k, v)
        self.k, self.v = kv4.held(k.double().numpy()), kv4.held(v.double().numpy())
        sdpa.attn_kv4_append(k.cuda(), v.cuda(), _i32(self.at.tolist()), self.pool, self.table, _i32([0] * len(lens)))
        self.cu = np.cumsum([0] + list(nodes))
        rows = int(self.cu[-1]) + extra_rows
        self.q = torch.randn((rows, H, d), generator=gen).to(torch.bfloat16).cuda()
        self.par = None if chain else _parents(rng, nodes) + [0] * extra_rows

    def call(self, **kw):
        args = _i32(self.cu.tolist()), None if self.par is None else _i32(self.par), _i32(self.lens)
        torch.cuda.current_stream().synchronize()
        self.alive = getattr(self, "alive", []) + [args]  # a call on another stream may still read them
        return _sdpa().sdpa_tree_kv4(self.q, args[0], args[1], self.pool, self.table, args[2], **kw)

    def check(self, o, lse, **kw):
        q, o, lse = self.q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, L in enumerate(self.lens):
            r, t = slice(int(self.cu[b]), int(self.cu[b + 1])), slice(int(self.at[b]), int(self.at[b + 1]))
            par = None if self.par is None else self.par[r]
            ro, rl, a, mag = tree.attention(q[r], self.k[t], self.v[t], L, par, **kw)
            bound = 2.0 ** -8 * (a + np.abs(ro)) + 2.0 ** -14 * a
            err = np.abs(o[r] - ro)
            assert np.all(err <= bound), f"sequence {b}: o off by {np.max(err - bound)} more than its bound"
            fin = np.isfinite(rl)
            assert np.array_equal(lse[:, r][~fin], rl[~fin])
            tol = 2.0 ** -17 * mag + 2.0 ** -18 * (1 + np.abs(np.where(fin, rl, 0)))
            assert np.all(np.abs(lse[:, r] - rl)[fin] <= tol[fin]), f"sequence {b}: lse"


CASES = [  # lens, nodes, H, H_kv, d, page
    ([0], [1], 1, 1, 64, 16),
    ([200], [7], 8, 2, 64, 16),
    ([1, 0, 127, 128, 129, 255], [3, 5, 1, 130, 8, 2], 4, 2, 128, 32),
    ([300, 5, 64], [40, 0, 33], 8, 1, 128, 64),          # one kv head: 320 rows of it
    ([77, 500, 130], [12, 1, 64], 6, 2, 64, 128),
    ([1500], [3], 3, 3, 128, 128),
    ([2, 700], [65, 20], 14, 2, 128, 16),                 # 7 heads a group: rows of no power of two
    ([400, 10, 0, 129, 77, 1000], [30, 1, 1, 1, 1, 1], 1, 1, 64, 16),   # 6 rows a sequence on average, 30 of one
    ([400, 10, 0, 129, 77], [20, 1, 1, 1, 1], 4, 2, 128, 32),           # 10 on average, 40 of one
    ([40, 3000, 256], [9, 2, 6], 15, 3, 128, 64),                       # 28 on average, 45 of one
    ([127, 2000], [3, 8], 6, 2, 64, 128),
]


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("lens,nodes,H,H_kv,d,page", CASES)
def test_tree_parity(lens, nodes, H, H_kv, d, page, chain):
    t = Trees(lens, nodes, H, H_kv, d, page, seed=len(lens) + d, chain=chain)
    o, lse = t.call()
    _clean()
    t.check(o, lse)


@pytest.mark.parametrize("nodes", [[1, 1, 1], [3, 0, 2]])
@pytest.mark.parametrize("G", [257, 300, 513])
def test_more_heads_a_kv_head_than_rows_of_a_block(G, nodes):
    """One node's heads span several blocks of rows."""
    t = Trees([130, 0, 64], nodes, G, 1, 64, 32, seed=G)
    o, lse = t.call()
    _clean()
    t.check(o, lse)


# heads a kv head such that a sequence has 8, 16, 32, 128 and more rows on average (32: a tile as well): the kernels' forms
@pytest.mark.parametrize("G", [1, 2, 4, 14, 40])
@pytest.mark.parametrize("window", [0, 1, 3, 50, 128, 300, 2 ** 31 - 1])
def test_windows(window, G):
    lens, nodes = [0, 40, 333, 128, 700, 510], [9, 8, 7, 1, 12, 4]
    t = Trees(lens, nodes, 2 * G, 2, 64 if window % 2 else 128, 16, seed=window % 97)
    o, lse = t.call(window=window)
    _clean()
    t.check(o, lse, window=window)


@pytest.mark.parametrize("window", [0, 1, 3, 50, 128, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("sink", ["vanilla", "off_by_one", "learnable"])
def test_windows_and_sinks(window, sink):
    lens, nodes, H = [0, 40, 333, 128, 700], [9, 30, 17, 1, 70], 4
    t = Trees(lens, nodes, H, 2, 64, 16, seed=window % 97)
    off = torch.linspace(-2, 3, H, device="cuda") if sink == "learnable" else None
    o, lse = t.call(window=window, softmax_type=sink, softmax_offset=off, scale=0.2)
    _clean()
    ref = None if sink == "vanilla" else np.zeros(H) if sink == "off_by_one" else off.double().cpu().numpy()
    t.check(o, lse, window=window, sink=ref, scale=float(np.float32(0.2)))


@pytest.mark.parametrize("window", [-1, 150])
def test_many_sequences(window):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 300, 90).tolist()
    nodes = rng.integers(0, 9, 90).tolist()
    t = Trees(lens, nodes, 4, 2, 64, 32, seed=5)
    o, lse = t.call(window=window)
    _clean()
    t.check(o, lse, window=window)


@pytest.mark.parametrize("nodes,H", [([33, 2], 4), ([4, 1], 3), ([9, 2], 2), ([9, 3], 4), ([60, 9], 8)])
def test_long_context_is_split(nodes, H):
    """A long prefix (its units spread over many CTAs) with a large score in one far token."""
    def edit(t, k, v):
        k[77] *= 4.0
    t = Trees([20000, 3], nodes, H, 1, 128, 64, seed=9, edit=edit)
    o, lse = t.call()
    _clean()
    t.check(o, lse)


@pytest.mark.parametrize("H,window", [(1, -1), (4, 300)])
def test_a_long_chain(H, window):
    """A prompt's continuation over a cached prefix: several row blocks, each up to its own last token."""
    t = Trees([333, 0], [700, 130], H, 1, 64, 64, seed=4, chain=True)
    o, lse = t.call(window=window)
    _clean()
    t.check(o, lse, window=window)


def test_no_sequences():
    sdpa = _sdpa()
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    pool = sdpa.kv4_pool(1, 2, 64, 16)
    o, lse = sdpa.sdpa_tree_kv4(q, _i32([0]), None, pool, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), _i32([]))
    assert torch.all(o == 0) and torch.all(lse == -np.inf)
    o, lse = sdpa.sdpa_tree_kv4(q[:0], _i32([0, 0]), None, pool, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), _i32([5]))
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    _clean()


def test_a_chain_equals_the_decode_of_the_newest_tokens():
    sdpa = _sdpa()
    lens, n = [130, 64, 1000], 3
    t = Trees(lens, [n] * 3, 8, 2, 128, 64, seed=2, chain=True)
    o, lse = t.call(window=200)
    o2, lse2 = sdpa.sdpa_decode_kv4(t.q.view(3, n, 8, 128), t.pool, t.table, _i32([L + n for L in lens]), window=200)
    t.check(o2.view(-1, 8, 128), lse2.permute(1, 0, 2).reshape(8, -1), window=200)
    t.check(o, lse, window=200)


def test_rows_of_no_sequence():
    sdpa = _sdpa()
    t = Trees([50, 10], [4, 3], 4, 2, 64, 16, extra_rows=3)
    o, lse = t.call()
    assert torch.all(o[7:] == 0) and torch.all(lse[:, 7:] == -np.inf)
    t.check(o, lse)
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    sdpa.attn_kv4_tree(t.q, _i32(t.cu.tolist()), _i32(t.par), t.pool, t.table, _i32(t.lens), o2, lse2)
    assert torch.all(o2[7:] == 7) and torch.all(lse2[:, 7:] == 7)
    assert torch.equal(o2[:7], o[:7]) and torch.equal(lse2[:, :7], lse[:, :7])
    o3 = torch.full_like(o, 7.0)
    sdpa.attn_kv4_tree(t.q, _i32(t.cu.tolist()), _i32(t.par), t.pool, t.table, _i32(t.lens), o3)  # no lse
    assert torch.equal(o3[:7], o[:7])
    _clean()


def test_parents_out_of_range_are_roots():
    t = Trees([20], [6], 2, 1, 64, 16)
    t.par = [-7, 0, 2, 9, 1, 2 ** 31 - 1]
    o, lse = t.call()
    t.check(o, lse)
    _clean()


@pytest.mark.parametrize("H", [2, 4, 8, 16, 64])  # 6 to 192 rows a kv head
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("side", ["k", "v"])
def test_nan_tokens_reach_only_their_descendants(side, d, H):
    """Node 1 and a prefix token before the window are NaN (held as NaN in 16 dims): nodes that do not see
    them are exact; those that do get NaN, for a value in its dims, for a key everywhere."""
    L, n = 140, 6
    par = [-1, 0, 0, 1, 2, -1]

    def edit(t, k, v):
        x = k if side == "k" else v
        x[L + 1, :, 20] = float("nan")
        x[3, :, 20] = float("inf")

    t = Trees([L], [n], H, 2, d, 16, edit=edit)
    t.par = par
    o, lse = t.call(window=100)
    _clean()
    sees = np.array([1 in tree.path(par, i) for i in range(n)])
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    dims = np.arange(d) // 16 == 1
    if side == "k":
        assert np.isnan(o[sees]).all() and np.isnan(lse[:, sees]).all()
    else:
        assert np.isnan(o[sees][:, :, dims]).all() and np.isfinite(o[sees][:, :, ~dims]).all()
        assert np.isfinite(lse).all()
    assert np.isfinite(o[~sees]).all() and np.isfinite(lse[:, ~sees]).all()
    k, v = np.nan_to_num(t.k), np.nan_to_num(t.v)
    ro, rl, a, _ = tree.attention(t.q.double().cpu().numpy(), k, v, L, par, window=100)
    ok = ~sees
    assert np.all(np.abs(o[ok] - ro[ok]) <= 2.0 ** -8 * (a[ok] + np.abs(ro[ok])) + 2.0 ** -14 * a[ok])


@pytest.mark.parametrize("H", [2, 10, 30, 100])
def test_a_nan_prefix_token_reaches_every_node(H):
    def edit(t, k, v):
        v[10, :, 0] = float("nan")
    t = Trees([300], [3], H, 1, 64, 64, edit=edit)
    o, lse = t.call()
    assert torch.isnan(o[:, :, :16]).all() and torch.isfinite(o[:, :, 16:]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("H", [4, 12, 40, 160])
def test_nan_query_rows_stay_alone(H):
    t = Trees([200], [4], H, 2, 128, 64)
    t.q[2, 1, 5] = float("nan")
    o, lse = t.call()
    bad = torch.isnan(o).all(-1)
    assert bad[2, 1] and torch.isnan(lse[1, 2]) and int(bad.sum()) == 1 and int(torch.isnan(lse).sum()) == 1


@pytest.mark.parametrize("H", [1, 2, 6, 20, 60])
def test_missing_pages_read_as_zeros(H):
    sdpa = _sdpa()
    t = Trees([100], [5], H, 1, 64, 16)
    t.table[0, 2] = -1
    t.table[0, 4] = 10 ** 6
    o, lse = t.call()
    torch.cuda.synchronize()
    st, site = sdpa.attn_last_device_error()
    assert st == 7 and site == 4
    for a, z in ((32, 48), (64, 80)):
        t.k[a:z] = t.v[a:z] = 0
    t.check(o, lse)
    t.lens = [90]   # pages before a window are not looked up
    t.k, t.v = t.k[:95], t.v[:95]
    t.at = np.array([0, 95])
    o, lse = t.call(window=9)
    _clean()
    t.check(o, lse, window=9)


@pytest.mark.parametrize("H", [1, 2, 4, 9, 40])
def test_tokens_past_the_table_do_not_exist(H):
    t = Trees([60], [8], H, 1, 64, 16)
    t.table = t.table[:, :4].contiguous()   # 64 tokens: nodes 4.. have no token
    o, lse = t.call()
    _clean()
    t.k, t.v = t.k[:64], t.v[:64]
    t.check(o, lse)
    t.table = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    o, lse = t.call()
    assert torch.all(o == 0) and torch.all(lse == -np.inf)
    o, lse = t.call(softmax_type="off_by_one")
    assert torch.all(o == 0) and torch.all(lse == 0)
    _clean()


def test_reproducible_two_streams_and_a_captured_graph():
    sdpa = _sdpa()
    a, b = Trees([900, 33], [20, 9], 8, 2, 128, 64, seed=1), Trees([500], [50], 4, 4, 64, 16, seed=2)
    ra, rb = a.call(), b.call()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    out = []
    for _ in range(8):
        out.append((a.call(stream=s1), b.call(stream=s2)))
    torch.cuda.synchronize()
    for x, y in out:
        assert all(torch.equal(p, q) for p, q in zip(x + y, ra + rb))
    cu, par, lens = _i32(a.cu.tolist()), _i32(a.par), _i32(a.lens)
    ws = torch.empty(sdpa.attn_kv4_tree_workspace_size(2, 29, 8, 2, 128), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    o, lse = torch.empty_like(ra[0]), torch.empty_like(ra[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sdpa.attn_kv4_tree(a.q, cu, par, a.pool, a.table, lens, o, lse, workspace=ws)
    lens.sub_(100)
    lens.clamp_(min=0)
    g.replay()
    want = sdpa.sdpa_tree_kv4(a.q, cu, par, a.pool, a.table, lens)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    _clean()


def test_cache_past_4_gb():
    """Page offsets past 32 bits: the last pages of a pool of 5 GB."""
    sdpa = _sdpa()
    page, H_kv, d = 128, 8, 128
    block = sdpa.kv4_block_bytes(page, d)
    n_pages = 5 * 2 ** 30 // (H_kv * block)
    pool = torch.empty((n_pages, H_kv, block), dtype=torch.uint8, device="cuda")
    table = _i32([[n_pages - 1, n_pages - 2]])
    gen = torch.Generator().manual_seed(0)
    k, v = (torch.randn((140, H_kv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    sdpa.attn_kv4_append(k.cuda(), v.cuda(), _i32([0, 140]), pool, table, _i32([0]))
    q = torch.randn((10, H_kv, d), generator=gen).to(torch.bfloat16).cuda()
    par = [-1, 0, 0, 1, 1, 2, 3, -1, 7, 8]
    o, lse = sdpa.sdpa_tree_kv4(q, _i32([0, 10]), _i32(par), pool, table, _i32([130]))
    ro, rl, a, mag = tree.attention(q.double().cpu().numpy(), kv4.held(k.double().numpy()), kv4.held(v.double().numpy()), 130,
                                    par)
    assert np.all(np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * (a + np.abs(ro)) + 2.0 ** -14 * a)
    sdpa.attn_kv4_keep(pool, table, _i32([130]), _i32([[0, 2, 5]]), d)
    gk, gv = sdpa.kv4_gather(pool, table, _i32([0, 3]), _i32([130]), 3, d)
    assert np.array_equal(gk.double().cpu().numpy(), kv4.held(k.double().numpy())[[130, 132, 135]])
    assert np.array_equal(gv.double().cpu().numpy(), kv4.held(v.double().numpy())[[130, 132, 135]])
    _clean()


# ------------------------------------------------------------------------------------------ accepted nodes


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layers", [1, 3])
def test_keep_moves_whole_tokens(page, d, layers):
    """Ascending, unsorted, repeated and empty lists, across pages; every other byte stays."""
    sdpa = _sdpa()
    rng = np.random.default_rng(page + d + layers)
    H, lens = 3, [0, 13, 16, 100, 127, 5]
    kept = [[0, 2, 3, 9, 11, 12, 20], [5, -1, 3, 1, 1, 1, 1], [-1] * 7, [6, 5, 4, 3, 2, 1, 0], [1, 1, 1, 0, 0, 0, 30],
            [0, 1, 2, 3, 4, 6, -4]]
    need = [-(-(L + 32) // page) for L in lens]
    n_pages = sum(need)
    perm = rng.permutation(n_pages)
    tab = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        tab[b, :m] = perm[at:at + m]
        at += m
    shape = (layers, n_pages, H, sdpa.kv4_block_bytes(page, d))
    pool = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).cuda()
    ref = pool.cpu().numpy().copy()
    places = []
    for w in range(page):
        at = {kv4.k_code_at(w, x, page, d)[0] for x in range(d)} | {kv4.v_code_at(w, x, page, d)[0] for x in range(d)}
        at |= {f(w, g, page, d) for g in range(d // 16) for f in (kv4.k_scale_at, kv4.v_scale_at)}
        places.append(at)
    # bytes of a token in the order of (part, dim): the same position in every token
    def order(w):
        return np.array([kv4.k_code_at(w, x, page, d)[0] for x in range(0, d, 2)] +
                        [kv4.v_code_at(w, x, page, d)[0] for x in range(0, d, 2)] +
                        [kv4.k_scale_at(w, g, page, d) for g in range(d // 16)] +
                        [kv4.v_scale_at(w, g, page, d) for g in range(d // 16)])
    orders = [order(w) for w in range(page)]
    assert all(set(o.tolist()) == p for o, p in zip(orders, places))
    for b, L in enumerate(lens):
        for i, a in enumerate(kept[b]):
            if a < 0:
                break
            s, t = L + a, L + i
            ref[:, tab[b, t // page], :, orders[t % page]] = ref[:, tab[b, s // page], :, orders[s % page]]
    view = pool if layers > 1 else pool[0]
    sdpa.attn_kv4_keep(view, _i32(tab.tolist()), _i32(lens), _i32(kept), d)
    _clean()
    assert np.array_equal(pool.cpu().numpy(), ref)


@pytest.mark.parametrize("order", ["ascending", "any"])
def test_keep_of_many_entries(order):
    """More entries than are looked up at once, against the moves one after another on whole tokens."""
    sdpa = _sdpa()
    rng = np.random.default_rng(7)
    page, d, H, L, n = 32, 64, 2, 45, 150
    k, v = (torch.from_numpy(rng.standard_normal((L + n, H, d))).to(torch.bfloat16) for _ in range(2))
    need = -(-(L + n) // page)
    pool = sdpa.kv4_pool(need, H, d, page).fill_(0xFF)
    table = _i32([rng.permutation(need).tolist()])
    sdpa.attn_kv4_append(k.cuda(), v.cuda(), _i32([0, L + n]), pool, table, _i32([0]))
    kept = (np.sort(rng.permutation(n)[:97]) if order == "ascending" else rng.integers(0, n, 97)).tolist()
    toks = list(range(L + n))
    tree.keep(toks, L, kept)
    sdpa.attn_kv4_keep(pool, table, _i32([L]), _i32([kept + [-1] * 3]), d)
    gk, gv = sdpa.kv4_gather(pool, table, _i32([0, L + n]), _i32([0]), L + n, d)
    _clean()
    assert np.array_equal(gk.double().cpu().numpy(), kv4.held(k.double().numpy())[toks])
    assert np.array_equal(gv.double().cpu().numpy(), kv4.held(v.double().numpy())[toks])


def test_keep_without_a_page():
    sdpa = _sdpa()
    pool = torch.randint(0, 256, (2, 1, sdpa.kv4_block_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    before = pool.clone()
    sdpa.attn_kv4_keep(pool, _i32([[0, -1, 1]]), _i32([15]), _i32([[3, 20]]), 64)  # sources in the missing page; then past it
    torch.cuda.synchronize()
    st, site = sdpa.attn_last_device_error()
    assert st == 7 and site == 5
    assert torch.equal(pool, before)
    sdpa.attn_kv4_keep(pool, _i32([[0, 1]]), _i32([2 ** 31 - 5]), _i32([[7]]), 64)  # token numbers past 31 bits
    torch.cuda.synchronize()
    assert sdpa.attn_last_device_error()[0] == 7 and torch.equal(pool, before)


def test_a_drafting_step():
    """Draft, append rotated, attend, keep an accepted path, go on: the cache then is that of the accepted tokens
    alone, and so is the next attention."""
    sdpa = _sdpa()
    H, Hk, d, page = 8, 2, 128, 16
    lens, nodes = [37, 90], [7, 5]
    pars = [[-1, 0, 0, 1, 2, 4, -1], [-1, 0, 1, 0, 3]]
    path = [[0, 2, 4, 5], [0, 3]]
    gen = torch.Generator().manual_seed(0)
    mk = lambda t, h: torch.randn((t, h, d), generator=gen).to(torch.bfloat16).cuda()
    table = _i32([[4, 1, 7, 0, 9, 11, 3], [2, 5, 6, 8, 10, 12, 13]])
    inv, gain = sdpa.rope_frequencies(d)
    cu0 = _i32([0, 37, 127])
    k0, v0 = mk(127, Hk), mk(127, Hk)
    pos0 = _i32(list(range(37)) + list(range(90)))
    t0 = sdpa.rope_table(inv, pos0, gain=gain)
    q1, k1, v1 = mk(12, H), mk(12, Hk), mk(12, Hk)
    depth = [len(tree.path(p, i)) - 1 for p in pars for i in range(len(p))]
    pos1 = _i32([L + dd for L, dd in zip([37] * 7 + [90] * 5, depth)])
    t1 = sdpa.rope_table(inv, pos1, gain=gain)
    pools = [sdpa.kv4_pool(14, Hk, d, page).fill_(0xFF) for _ in range(2)]
    for p in pools:
        sdpa.kv4_append_rope(None, k0, v0, t0, cu0, p, table, _i32([0, 0]))
    cu1 = _i32([0, 7, 12])
    qr = sdpa.kv4_append_rope(q1, k1, v1, t1, cu1, pools[0], table, _i32(lens))
    o, lse = sdpa.sdpa_tree_kv4(qr, cu1, _i32(pars[0] + pars[1]), pools[0], table, _i32(lens))
    sdpa.attn_kv4_keep(pools[0], table, _i32(lens), _i32([path[0], path[1] + [-1, -1]]), d)
    # the accepted tokens alone
    rows = torch.tensor(path[0] + [7 + i for i in path[1]], device="cuda")
    cu2 = _i32([0, 4, 6])
    q2 = sdpa.kv4_append_rope(q1[rows], k1[rows], v1[rows], t1[rows].contiguous(), cu2, pools[1], table, _i32(lens))
    o2, lse2 = sdpa.sdpa_tree_kv4(q2, cu2, None, pools[1], table, _i32(lens))
    new = [41, 92]
    ks = [sdpa.kv4_gather(p, table, _i32([0, 41, 133]), _i32([0, 0]), 133, d) for p in pools]
    assert torch.equal(ks[0][0], ks[1][0]) and torch.equal(ks[0][1], ks[1][1])
    # the path's nodes saw the same tokens in the tree as in the chain; the order of their sums may differ
    a, b = o[rows].double(), o2.double()
    vmax = float(ks[0][1].abs().double().max())
    assert float((a - b).abs().max()) <= 2 * 2.0 ** -7 * vmax
    assert float((lse[:, rows] - lse2).abs().max()) <= 2.0 ** -10
    q3 = mk(2, H)
    outs = [sdpa.sdpa_tree_kv4(q3, _i32([0, 1, 2]), None, p, table, _i32([n - 1 for n in new])) for p in pools]
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    _clean()


def test_refusals():
    sdpa = _sdpa()
    t = Trees([20], [3], 4, 2, 64, 16)
    cu, par, lens = _i32([0, 3]), _i32(t.par), _i32([20])
    with pytest.raises(TypeError):
        sdpa.sdpa_tree_kv4(t.q.half(), cu, par, t.pool, t.table, lens)
    with pytest.raises(ValueError):
        sdpa.sdpa_tree_kv4(t.q, cu, par[:2].contiguous(), t.pool, t.table, lens)
    with pytest.raises(ValueError):
        sdpa.sdpa_tree_kv4(t.q, _i32([0, 1, 3]), par, t.pool, t.table, lens)
    with pytest.raises(ValueError):
        sdpa.sdpa_tree_kv4(t.q[:, :, :32].contiguous(), cu, par, t.pool, t.table, lens)
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_tree_kv4(t.q[:, :3].contiguous(), cu, par, t.pool, t.table, lens)  # 3 heads over 2 kv heads
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_tree_kv4(t.q, cu, par, t.pool, t.table, lens,
                           workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sdpa.attn_kv4_tree(t.q, cu, par, t.pool, t.table, lens, torch.empty_like(t.q)[:2])
    with pytest.raises(ValueError):
        sdpa.attn_kv4_keep(t.pool, t.table, lens, _i32([[0], [1]]), 64)
    with pytest.raises(TypeError):
        sdpa.attn_kv4_keep(t.pool, t.table, lens, torch.zeros((1, 2), dtype=torch.int64, device="cuda"), 64)
