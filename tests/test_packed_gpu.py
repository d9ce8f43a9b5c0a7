"""Attention over packed sequences on the GPU against the fp64 oracle, one sequence at a time:
ragged lengths, sequences without queries or keys, masks, sinks, offsets that are not
offsets, isolation of neighbours, and the differentiable form.  Tolerances are those of
every other parity test (O max-abs 2e-2, LSE 1e-3, gradients relative L2 1e-2)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import LEARNABLE, OFF_BY_ONE, VANILLA
from parity_util import TOL_GRAD, TOL_LSE, TOL_O, rel_l2

pytestmark = pytest.mark.gpu


def _sdpa():
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + np.cumsum(lens).tolist())


def _clean():
    torch.cuda.synchronize()
    st, site = _sdpa().attn_last_device_error()
    assert st == 0, f"device error status {st} site {site:#x}"


def _inputs(lq, lk, H, H_kv, dqk, dv, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    Tq, Tk = sum(lq) + extra, sum(lk) + extra
    return dict(q=r(Tq, H, dqk), k=r(Tk, H_kv, dqk), v=r(Tk, H_kv, dv), dout=r(Tq, H, dv), off=torch.randn(H, generator=g))


def _reference(x, lq, lk, **kw):
    """Every sequence on its own through the oracle."""
    st = kw["softmax_type"]
    off = x["off"].double().numpy() if st == LEARNABLE else None
    H, dv = x["q"].shape[1], x["v"].shape[2]
    o = np.zeros((sum(lq), H, dv))
    lse = np.zeros((H, sum(lq)))
    dq, dk, dvv = (np.zeros(tuple(x[n].shape)) for n in "qkv")
    d_off = np.zeros(H)
    a = c = 0
    for n, m in zip(lq, lk):
        q, k, v, do = (x[t][s].double().numpy()[None] for t, s in
                       (("q", slice(a, a + n)), ("k", slice(c, c + m)), ("v", slice(c, c + m)), ("dout", slice(a, a + n))))
        if n and m:
            f = oracle.attention_fwd(q, k, v, offset=off, scale=None, **kw)
            g = oracle.attention_bwd(q, k, v, do, offset=off, scale=None, **kw)
            o[a:a + n], lse[:, a:a + n] = f["o"][0], f["lse"][0]
            dq[a:a + n], dk[c:c + m], dvv[c:c + m] = g["dq"][0], g["dk"][0], g["dv"][0]
            if st == LEARNABLE:
                d_off += g["d_offset"]
        elif n:
            lse[:, a:a + n] = {VANILLA: np.full(H, -np.inf), OFF_BY_ONE: np.zeros(H), LEARNABLE: off}[st][:, None]
        a, c = a + n, c + m
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dvv, d_offset=d_off)


def _run(x, cu_q, cu_kv, *, causal, window, softmax_type):
    sdpa = _sdpa()
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "dout"))
    off = x["off"].cuda() if softmax_type == LEARNABLE else None
    kw = dict(causal=causal, window=window, softmax_type=softmax_type, softmax_offset=off)
    o, lse = sdpa.sdpa_forward_packed(q, k, v, cu_q, cu_kv, **kw)
    dq, dk, dv, d_off = sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu_q, cu_kv, **kw)
    _clean()
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, d_offset=d_off)


def _compare(got, ref, what):
    g = {n: t.double().cpu().numpy() for n, t in got.items() if t is not None}
    n, m = ref["o"].shape[0], ref["dk"].shape[0]
    assert np.abs(g["o"][:n] - ref["o"]).max(initial=0) <= TOL_O, what
    fin = np.isfinite(ref["lse"])
    assert np.array_equal(g["lse"][:, :n][~fin], ref["lse"][~fin]), what
    assert np.abs(g["lse"][:, :n][fin] - ref["lse"][fin]).max(initial=0) <= TOL_LSE, what
    for t, rows in (("dq", n), ("dk", m), ("dv", m)):
        e = rel_l2(g[t][:rows], ref[t][:rows])
        assert e <= TOL_GRAD, f"{what}: {t} relative L2 {e}"


# name, lens_q, lens_kv (None: the same), H_q, H_kv, d_qk, d_v, causal, window, softmax type
CASES = [
    ("gqa_d128", [300, 1, 128, 129, 17, 256, 511], None, 8, 2, 128, 128, True, -1, VANILLA),
    ("gqa_d64_window_learnable", [130, 257, 5, 64, 400], None, 8, 2, 64, 64, True, 50, LEARNABLE),
    ("mla", [200, 70, 129, 1], None, 4, 4, 192, 128, True, -1, OFF_BY_ONE),
    ("mla_learnable_cross", [100, 0, 33], [260, 40, 0], 4, 2, 192, 128, False, -1, LEARNABLE),
    ("mha_noncausal", [190, 5, 133], None, 4, 4, 128, 128, False, -1, VANILLA),
    ("mqa_d64", [257, 100, 64], None, 8, 1, 64, 64, True, -1, OFF_BY_ONE),
    ("group7_d128", [140, 1, 1, 260], None, 7, 1, 128, 128, True, 20, LEARNABLE),
    ("cross_lengths", [40, 300, 0, 1, 128], [256, 100, 70, 1, 0], 8, 2, 128, 128, True, -1, LEARNABLE),
    ("cross_noncausal_empty", [0, 64, 10], [5, 0, 300], 4, 2, 64, 64, False, -1, VANILLA),
    ("no_keys_at_all", [5, 130], [0, 0], 4, 2, 128, 128, True, -1, OFF_BY_ONE),
    ("no_queries_at_all", [0, 0], [5, 130], 4, 2, 128, 128, True, -1, LEARNABLE),
    ("single_tokens", [1] * 40, None, 4, 2, 64, 64, True, -1, VANILLA),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_parity(case):
    name, lq, lk, H, H_kv, dqk, dv, causal, window, st = case
    x = _inputs(lq, lk or lq, H, H_kv, dqk, dv, seed=len(name))
    kw = dict(causal=causal, window=window, softmax_type=st)
    got = _run(x, _cu(lq), _cu(lk) if lk else None, **kw)
    ref = _reference(x, lq, lk or lq, **kw)
    _compare(got, ref, name)
    again = _run(x, _cu(lq), _cu(lk) if lk else None, **kw)
    for n, t in got.items():
        assert t is None or torch.equal(t, again[n]), f"{name}: {n} is not reproducible"
    if st == LEARNABLE:
        # fp32 rounding only.  With A_i = sum_j P_ij |dP_ij| and p_i = exp(off - LSE_i), each
        # term p_i D*_i is off by a small multiple of the scores' fp32 error, 2^-17 sum_x |q_x k_x|
        # scale (at most 16 or so here), times p_i (A_i + |D_i|): 2^-13 of it in all.
        bound = np.zeros(H)
        a = c = 0
        for n, m in zip(lq, lk or lq):
            for h in range(H):
                q, do = (x[t][a:a + n, h].double().numpy() for t in ("q", "dout"))
                k, v = (x[t][c:c + m, h // (H // H_kv)].double().numpy() for t in ("k", "v"))
                i, j = np.arange(n)[:, None], np.arange(m)[None, :]
                vis = (j <= i) & ((window < 0) | (j >= i - window)) if causal else np.ones((n, m), bool)
                s = np.where(vis, q @ k.T / np.sqrt(dqk), -np.inf)
                p = np.exp(s - ref["lse"][h, a:a + n][:, None])
                dp = do @ v.T
                A = (p * np.abs(dp)).sum(1)
                D = np.abs((do * ref["o"][a:a + n, h]).sum(1))
                bound[h] += (np.exp(x["off"][h].double().item() - ref["lse"][h, a:a + n]) * (A + D)).sum() if n else 0
            a, c = a + n, c + m
        err = np.abs(got["d_offset"].double().cpu().numpy() - ref["d_offset"])
        assert np.all(err <= 2.0 ** -13 * bound), f"{name}: d_offset off by {err}, bound {2.0 ** -13 * bound}"


def test_forward_equals_the_plain_call_bit_for_bit():
    sdpa = _sdpa()
    lens = [300, 64, 1, 513]
    x = _inputs(lens, lens, 8, 2, 128, 128, 3)
    o, lse = sdpa.sdpa_forward_packed(*(x[n].cuda() for n in "qkv"), _cu(lens), window=100)
    at = 0
    for n in lens:
        q, k, v = (x[t][at:at + n].cuda()[None].contiguous() for t in "qkv")
        a, b = sdpa.sdpa_forward(q, k, v, window=100)
        assert torch.equal(o[at:at + n], a[0]) and torch.equal(lse[:, at:at + n], b[0])
        at += n
    _clean()


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("what", ["k", "v", "q", "dout"])
def test_infinities_and_nans_stay_in_their_sequence(dims, what):
    """A sequence of NaN and infinities between two others changes no bit of theirs (their last
    tiles reach into it), nor do rows of no sequence."""
    lens = [70, 100, 200]
    x = _inputs(lens, lens, 4, 2, *dims, seed=7, extra=60)
    cu = _cu(lens)
    kw = dict(causal=True, window=-1, softmax_type=LEARNABLE)
    base = _run(x, cu, None, **kw)
    y = dict(x)
    y[what] = x[what].clone()
    y[what][70:170] = float("nan")
    y[what][75:165:2] = float("inf")
    y[what][370:] = float("nan")
    got = _run(y, cu, None, **kw)
    keep = list(range(70)) + list(range(170, 370))
    for n in ("o", "dq", "dk", "dv"):
        assert torch.isfinite(got[n][keep].float()).all(), n
        assert torch.equal(got[n][keep], base[n][keep]), n
    assert torch.equal(got["lse"][:, keep], base["lse"][:, keep])
    assert torch.all(got["o"][370:] == 0) and torch.all(got["dq"][370:] == 0) and torch.all(got["dk"][370:] == 0)


def test_rows_of_no_sequence_are_left_alone():
    sdpa = _sdpa()
    lens = [33, 130]
    x = _inputs(lens, lens, 4, 2, 64, 64, 11, extra=45)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "dout"))
    T = q.shape[0]
    o, lse = torch.full_like(q, 5.0), torch.full((4, T), 5.0, device="cuda")
    g = [torch.full_like(t, 5.0) for t in (q, k, v)]
    cu = _cu(lens)
    sdpa.attn_fwd_packed(q, k, v, o, lse, cu)
    sdpa.attn_bwd_packed(q, k, v, o, do, lse, *g, None, cu)
    _clean()
    for t in (o, *g):
        assert torch.all(t[163:] == 5) and not torch.all(t[:163] == 5)
    assert torch.all(lse[:, 163:] == 5)
    a, b = sdpa.sdpa_forward_packed(q, k, v, cu)
    assert torch.equal(a[:163], o[:163]) and torch.all(a[163:] == 0) and torch.all(b[:, 163:] == -float("inf"))
    # no sequence at all, and no rows at all
    a, b = sdpa.sdpa_forward_packed(q, k, v, _i32([0]))
    g2 = sdpa.sdpa_backward_packed(q, k, v, a, do, b, _i32([0]))
    _clean()
    assert torch.all(a == 0) and all(torch.all(t == 0) for t in g2[:3])
    e = q[:0]
    a, b = sdpa.sdpa_forward_packed(e, k[:0], v[:0], _i32([0, 0, 0]))
    g2 = sdpa.sdpa_backward_packed(e, k[:0], v[:0], a, e, b, _i32([0, 0, 0]))
    _clean()
    assert a.shape[0] == 0 and g2[1].shape[0] == 0


def test_rows_before_the_first_sequence_and_huge_windows():
    sdpa = _sdpa()
    x = _inputs([100], [100], 4, 2, 128, 128, 12, extra=20)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "dout"))
    cu = _i32([30, 30, 100])
    o, lse = sdpa.sdpa_forward_packed(q, k, v, cu, window=2 ** 40)
    g = sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu, window=2 ** 31 - 1)
    part = [t[30:100].contiguous() for t in (q, k, v)]
    o1, lse1 = sdpa.sdpa_forward_packed(*part, _i32([0, 70]))
    g1 = sdpa.sdpa_backward_packed(*part, o1, do[30:100].contiguous(), lse1, _i32([0, 70]))
    _clean()
    assert torch.equal(o[30:100], o1) and torch.equal(lse[:, 30:100], lse1)
    for a, b in zip(g[:3], g1[:3]):
        assert torch.equal(a[30:100], b)
    for t in (o, *g[:3]):
        assert torch.all(t[:30] == 0) and torch.all(t[100:] == 0)
    assert torch.all(lse[:, :30] == -float("inf")) and torch.all(lse[:, 100:] == -float("inf"))


def test_offsets_that_are_not_offsets_are_clamped():
    """Not ascending, negative, past the end: each is clamped to [0, T] and to the running
    maximum, and nothing outside the tensors is touched."""
    raw = [-5, 40, 20, 300, 100, 9999]
    clean = [0, 40, 40, 200, 200, 200]
    lens = np.diff(clean).tolist()
    x = _inputs([200], [200], 4, 2, 128, 128, 13)
    kw = dict(causal=True, window=-1, softmax_type=VANILLA)
    a, b = _run(x, _i32(raw), None, **kw), _run(x, _cu(lens), None, **kw)
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("raw", [[0, 300, 300, 557, 558], [7, 100, 40, 612, 9999, 3], [-5, 0, 0, 640]])
def test_forward_with_and_without_a_plan_kernel(dims, raw):
    """A batch small enough for its blocks to find their tiles themselves, and the same one with
    empty sequences behind it until a plan kernel has to list them: every bit the same, rows of
    no sequence included; so with offsets of the keys' own."""
    sdpa = _sdpa()
    T, H, H_kv = 640, 4, 2
    x = _inputs([T], [T], H, H_kv, *dims, 5)
    q, k, v = (x[n].cuda() for n in "qkv")
    kv = [0] + [(3 * c) // 4 for c in raw[1:]]
    for cu_kv in (None, kv):
        for kw in (dict(window=70), dict(causal=False, softmax_type=OFF_BY_ONE)):
            many = lambda c: None if c is None else _i32(c + [c[-1]] * 40)
            few = lambda c: None if c is None else _i32(c)
            a = sdpa.sdpa_forward_packed(q, k, v, few(raw), few(cu_kv), **kw)
            b = sdpa.sdpa_forward_packed(q, k, v, many(raw), many(cu_kv), **kw)
            _clean()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (cu_kv, kw)
    lens = [0] * 30 + [T]  # the most sequences that need no plan kernel, and one more
    a, b = (sdpa.sdpa_forward_packed(q, k, v, _cu(n)) for n in (lens, [0] + lens))
    _clean()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dims", [(64, 64), (192, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences_with_and_without_keys(dims, causal):
    """More work tiles than blocks, of any cost: some sequences have no keys, some no queries, and
    a tile without keys follows one with keys in the same block."""
    g = np.random.default_rng(int(causal))
    lq = g.integers(0, 300, 90)
    lk = np.where(g.random(90) < 0.4, 0, g.integers(1, 400, 90))
    lq, lk = lq.tolist(), lk.tolist()
    x = _inputs(lq, lk, 4, 2, *dims, seed=23)
    kw = dict(causal=causal, window=-1, softmax_type=LEARNABLE)
    got, ref = _run(x, _cu(lq), _cu(lk), **kw), _reference(x, lq, lk, **kw)
    _compare(got, ref, f"{dims} causal={causal}")
    again = _run(x, _cu(lq), _cu(lk), **kw)
    for n, t in got.items():
        assert torch.equal(t, again[n]), n


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("window,lens_kv", [(0, None), (1, None), (5, None), (15, None), (16, None), (31, None),
                                            (-1, [3, 1, 9, 2]), (-1, [32, 17, 16, 31]), (40, [90, 60, 130, 20])])
def test_gradients_of_rows_that_see_few_keys(dims, window, lens_kv):
    """dS and the results are rounded to bf16.  A rounding is off by at most 2^-8 of a value, evenly
    over that step: 2^-8 / sqrt(3) for a mantissa of 1, with mantissas spread over [1, 2) 0.72 of
    it, 0.00163 relative L2; two of them 0.0023, and with a tenth more for samples of 10^4 values
    and the fp32 arithmetic 0.0026.  D from the stored bf16 O adds a third error of that size
    where rows see few keys, so they get it from fp32 scores."""
    lens = [150, 70, 201, 64]
    x = _inputs(lens, lens_kv or lens, 4, 2, *dims, seed=31)
    kw = dict(causal=True, window=window, softmax_type=OFF_BY_ONE)
    got = _run(x, _cu(lens), _cu(lens_kv) if lens_kv else None, **kw)
    ref = _reference(x, lens, lens_kv or lens, **kw)
    for n in ("dq", "dk"):
        e = rel_l2(got[n].double().cpu().numpy(), ref[n])
        assert e <= 0.0026, f"{n}: {e}"


def test_more_sequences_than_plan_threads_and_a_long_one():
    """3,000 short sequences around one of 5,000 rows; a sample of them against the oracle."""
    g = np.random.default_rng(1)
    lens = g.integers(0, 12, 3000).tolist()
    lens[1700] = 5000
    x = _inputs(lens, lens, 2, 1, 64, 64, 17)
    kw = dict(causal=True, window=-1, softmax_type=VANILLA)
    got = _run(x, _cu(lens), None, **kw)
    at = np.cumsum([0] + lens)
    for b in (0, 1, 1023, 1024, 1025, 1699, 1701, 2047, 2048, 2999):
        s = slice(int(at[b]), int(at[b + 1]))
        y = {n: x[n][s] for n in ("q", "k", "v", "dout")}
        ref = _reference(dict(y, off=x["off"]), [lens[b]], [lens[b]], **kw)
        _compare({n: (t[:, s] if n == "lse" else t[s]) for n, t in got.items() if n != "d_offset"}, ref, f"sequence {b}")
    s = slice(int(at[1700]), int(at[1701]))
    sdpa = _sdpa()
    o, lse = sdpa.sdpa_forward(*(x[n][s].cuda()[None].contiguous() for n in "qkv"))
    assert torch.equal(got["o"][s], o[0]) and torch.equal(got["lse"][:, s], lse[0])
    dq, dk, dv, _ = sdpa.sdpa_backward(*(x[n][s].cuda()[None].contiguous() for n in "qkv"), o, x["dout"][s].cuda()[None].contiguous(), lse)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert rel_l2(got[n][s].double().cpu().numpy(), t[0].double().cpu().numpy()) <= TOL_GRAD, n


def test_rows_past_2_to_31_elements():
    """530,000 rows of 32 heads of 128 (2.2e9 elements of q, o, dout, dq): the last sequences agree
    with the same sequences on their own."""
    sdpa = _sdpa()
    T, H, d = 530000, 32, 128
    lens = [400] * 1324 + [280, 120]
    g = torch.Generator("cuda").manual_seed(33)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, do, k, v = r(T, H, d), r(T, H, d), r(T, 1, d), r(T, 1, d)
    cu = _cu(lens)
    o, lse = sdpa.sdpa_forward_packed(q, k, v, cu)
    dq, dk, dv, _ = sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu)
    tail = slice(T - 400, T)
    part = [t[tail].contiguous() for t in (q, k, v)]
    cu2 = _cu([280, 120])
    o2, lse2 = sdpa.sdpa_forward_packed(*part, cu2)
    g2 = sdpa.sdpa_backward_packed(*part, o2, do[tail].contiguous(), lse2, cu2)
    _clean()
    assert torch.equal(o[tail], o2) and torch.equal(lse[:, tail], lse2)
    # (few tiles split the query heads of a group: another order of the fp32 sums)
    for a, b in zip((dq, dk, dv), g2):
        assert rel_l2(a[tail].double().cpu().numpy(), b.double().cpu().numpy()) <= TOL_GRAD


def test_gradients_against_differences():
    """The kernel's dq, dk, dv, d_offset against central differences of the oracle's fp64 forward
    along random directions u: |<grad, u> - difference| within the gradient tolerance of
    |grad| |u| / sqrt(n) times 8 (a random direction sees the error vector's projection,
    |error| |u| / sqrt(n) times a standard normal; h = 1e-4 leaves 1e-8 of third order)."""
    lens = [60, 131]
    H, H_kv = 4, 2
    x = _inputs(lens, lens, H, H_kv, 64, 64, 19)
    kw = dict(causal=True, window=30, softmax_type=LEARNABLE)
    got = _run(x, _cu(lens), None, **kw)
    xd = {n: t.double().numpy() for n, t in x.items()}

    def loss(z):
        total, a = 0.0, 0
        for n in lens:
            f = oracle.attention_fwd(z["q"][None, a:a + n], z["k"][None, a:a + n], z["v"][None, a:a + n],
                                     offset=z["off"], scale=None, **kw)
            total += (f["o"][0] * z["dout"][a:a + n]).sum()
            a += n
        return total

    rng = np.random.default_rng(2)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("off", "d_offset")):
        g = got[grad].double().cpu().numpy()
        for _ in range(3):
            u = rng.standard_normal(xd[name].shape)
            hi, lo = (dict(xd, **{name: xd[name] + e * u}) for e in (1e-4, -1e-4))
            diff = (loss(hi) - loss(lo)) / 2e-4
            tol = 8 * TOL_GRAD * np.linalg.norm(g) * np.linalg.norm(u) / np.sqrt(u.size)
            assert abs((g * u).sum() - diff) <= tol, f"{grad}: {(g * u).sum()} against {diff} (tolerance {tol})"


def test_autograd_and_cross_offsets():
    sdpa = _sdpa()
    lq, lk = [100, 30], [50, 140]
    x = _inputs(lq, lk, 4, 2, 64, 64, 23)
    leaf = {n: x[n].cuda().requires_grad_(True) for n in ("q", "k", "v", "off")}
    kw = dict(causal=False, softmax_type=LEARNABLE)
    o = sdpa.attention_packed(leaf["q"], leaf["k"], leaf["v"], _cu(lq), _cu(lk), leaf["off"], **kw)
    o.backward(x["dout"].cuda().transpose(0, 1).contiguous().transpose(0, 1))  # a gradient that is not contiguous
    got = _run(x, _cu(lq), _cu(lk), window=-1, **kw)
    assert torch.equal(o.detach(), got["o"])
    for n, g in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("off", "d_offset")):
        assert torch.equal(leaf[n].grad, got[g]), n


def test_calls_on_two_streams_at_once():
    """Forward and backward of two packed batches, many times over on two streams without waiting
    for each other, give the bits of the same calls one at a time."""
    sdpa = _sdpa()
    jobs = []
    for lens, dims, seed in (([300, 41, 700], (128, 128), 41), ([64, 512, 1, 130], (64, 64), 42)):
        x = _inputs(lens, lens, 4, 2, *dims, seed)
        jobs.append(([x[n].cuda() for n in ("q", "k", "v", "dout")], x["off"].cuda(), _cu(lens)))

    def step(job, stream=None):
        (q, k, v, do), off, cu = job
        kw = dict(softmax_type=LEARNABLE, softmax_offset=off, stream=stream)
        o, lse = sdpa.sdpa_forward_packed(q, k, v, cu, **kw)
        return (o, lse) + sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu, **kw)

    alone = [step(j) for j in jobs]
    _clean()
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(step(jobs[i], s))
    for s in streams:
        s.synchronize()
    _clean()
    for i in range(2):
        for res in got[i]:
            for a, b in zip(res, alone[i]):
                assert torch.equal(a, b)


def test_captured_graphs_and_another_stream():
    """Forward and backward captured twice, with workspaces of their own, replay on new offsets
    with the eager run's bits; and the eager run on a side stream has them too."""
    sdpa = _sdpa()
    T, H, H_kv, d = 600, 4, 2, 128
    x = _inputs([T], [T], H, H_kv, d, d, 29)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "dout"))
    off = x["off"].cuda()
    kw = dict(softmax_type=LEARNABLE, softmax_offset=off, zero_rest=True)
    sets = [[100, 200, 300], [600, 0, 0], [7, 350, 9]]

    def step(cu, out, ws):
        sdpa.attn_fwd_packed(q, k, v, out[0], out[1], cu, workspace=ws[0], **kw)
        sdpa.attn_bwd_packed(q, k, v, out[0], do, out[1], *out[2:], cu, workspace=ws[1], **kw)

    def buffers():
        out = [torch.empty_like(q), torch.empty((H, T), device="cuda"), torch.empty_like(q), torch.empty_like(k),
               torch.empty_like(v), torch.empty(H, device="cuda")]
        ws = [torch.empty(sdpa.attn_packed_workspace_size(3, T, T, H, H_kv, d, d, b), dtype=torch.uint8, device="cuda")
              for b in (False, True)]
        return out, ws

    eager = []
    side = torch.cuda.Stream()
    for lens in sets:
        out, ws = buffers()
        cu = _cu(lens)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(cu, out, ws)
        side.synchronize()
        eager.append(out)
    graphs = []
    for _ in range(2):
        out, ws = buffers()
        cu = _cu(sets[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(cu, out, ws)
        graphs.append((g, cu, out, ws))
    for i, lens in enumerate(sets):
        for j, (g, cu, out, _) in enumerate(graphs):
            cu.copy_(_cu(sets[(i + j) % 3]))
            g.replay()
        torch.cuda.synchronize()
        for j, (_, _, out, _) in enumerate(graphs):
            for a, b in zip(out, eager[(i + j) % 3]):
                assert torch.equal(a, b)
    _clean()


def test_refusals():
    sdpa = _sdpa()
    x = _inputs([20], [20], 4, 2, 64, 64, 1)
    q, k, v = (x[n].cuda() for n in "qkv")
    cu = _cu([20])
    bad = [(q.float(), k, v, cu), (q, k[:, :1].contiguous(), v, cu), (q, k, v, cu.long()), (q, k[:10], v[:10], cu),
           (q, k, v, cu, _cu([10, 10])), (q[:, :, ::2], k, v, cu), (q[None], k, v, cu), (q, k, v, cu[:0]),
           (q, k, v, cu.cpu())]
    for args in bad:
        with pytest.raises((TypeError, ValueError)):
            sdpa.sdpa_forward_packed(*args)
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_forward_packed(q, k, v, cu, causal=False, window=3)
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_forward_packed(q, k, v, cu, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sdpa.AttnError):
        sdpa.sdpa_forward_packed(q, k, v, cu, softmax_type=LEARNABLE)
    with pytest.raises(ValueError):
        sdpa.sdpa_forward_packed(q, k, v, cu, softmax_type=LEARNABLE, softmax_offset=torch.zeros(3, device="cuda"))


def test_prefill_of_a_continuation_over_a_cached_prefix():
    """The operators together: prompts attend packed and enter the 4-bit cache; the newest token's
    attention over the cache agrees with packed attention of that token over the gathered cache."""
    sdpa = _sdpa()
    lens, H, H_kv, d, page = [300, 17, 129], 8, 2, 128, 32
    x = _inputs(lens, lens, H, H_kv, d, d, 31)
    q, k, v = (x[n].cuda() for n in "qkv")
    sdpa.sdpa_forward_packed(q, k, v, _cu(lens))
    need = [-(-n // page) for n in lens]
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    pool, zero = sdpa.kv4_pool(at, H_kv, d, page), _i32([0, 0, 0])
    sdpa.attn_kv4_append(k, v, _cu(lens), pool, table.cuda(), zero)
    last = torch.tensor(np.cumsum(lens) - 1, device="cuda")
    o, lse = sdpa.sdpa_decode_kv4(q[last].unsqueeze(1).contiguous(), pool, table.cuda(), _i32(lens))
    kc, vc = sdpa.kv4_gather(pool, table.cuda(), _cu(lens), zero, sum(lens), d)
    o2, lse2 = sdpa.sdpa_forward_packed(q[last].contiguous(), kc, vc, _cu([1, 1, 1]), _cu(lens), causal=False)
    _clean()
    # both round P and o to bf16: each is within 2^-8 (sum P |v| + |o|) of the exact value
    bound = 2.0 ** -7 * (o2.float().abs() + vc.float().abs().max())
    assert torch.all((o[:, 0].float() - o2.float()).abs() <= bound)
    assert (lse[:, :, 0].t() - lse2).abs().max() <= TOL_LSE


def test_one_workspace_for_batches_after_another():
    """Work lists are written while the kernels that read them are already set up: forward and backward of
    batches with other offsets, one after another in the same workspaces, never see an earlier list."""
    sdpa = _sdpa()
    T, H, H_kv, d = 5000, 8, 2, 64
    x = _inputs([T], [T], H, H_kv, d, d, 47)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "dout"))
    off = x["off"].cuda()
    kw = dict(window=300, softmax_type=LEARNABLE, softmax_offset=off)
    rng = np.random.default_rng(3)
    batches = []
    for _ in range(6):
        cut = np.sort(rng.integers(0, T + 1, 39))
        batches.append(_i32([0] + cut.tolist() + [T]))
    alone = []
    for cu in batches:
        o, lse = sdpa.sdpa_forward_packed(q, k, v, cu, **kw)
        alone.append((o, lse) + sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu, **kw))
    ws = [torch.empty(sdpa.attn_packed_workspace_size(40, T, T, H, H_kv, d, d, b), dtype=torch.uint8, device="cuda")
          for b in (False, True)]
    got = []
    for i in range(30):
        cu = batches[i % 6]
        o, lse = sdpa.sdpa_forward_packed(q, k, v, cu, workspace=ws[0], **kw)
        got.append((o, lse) + sdpa.sdpa_backward_packed(q, k, v, o, do, lse, cu, workspace=ws[1], **kw))
    _clean()
    for i, res in enumerate(got):
        for a, b in zip(res, alone[i % 6]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
def test_lse_of_a_row_with_a_nan_score_is_nan(dims):
    """-inf would say that the row sees no key.  A query's NaN makes its own row's lse and o NaN, a key's
    those of the rows that see it; the other rows' lse is as without it."""
    sdpa = _sdpa()
    lens = [150, 300, 40]
    x = _inputs(lens, lens, 4, 2, *dims, seed=53)
    cu = _cu(lens)
    for st in (VANILLA, OFF_BY_ONE):
        base = sdpa.sdpa_forward_packed(*(x[n].cuda() for n in "qkv"), cu, softmax_type=st)
        q, k = x["q"].clone(), x["k"].clone()
        q[7, 1, 3] = q[449, 2, 60] = q[489, 0, 0] = float("nan")
        o, lse = sdpa.sdpa_forward_packed(q.cuda(), k.cuda(), x["v"].cuda(), cu, softmax_type=st)
        bad = torch.zeros((4, 490), dtype=torch.bool, device="cuda")
        bad[1, 7] = bad[2, 449] = bad[0, 489] = True
        _clean()
        assert torch.equal(torch.isnan(lse), bad) and torch.isnan(o[7, 1]).all()
        assert torch.equal(lse[~bad], base[1][~bad])
        k[150 + 133, 1, 5] = float("nan")  # key 133 of the second sequence, heads 2 and 3
        o, lse = sdpa.sdpa_forward_packed(x["q"].cuda(), k.cuda(), x["v"].cuda(), cu, softmax_type=st, window=90)
        base = sdpa.sdpa_forward_packed(*(x[n].cuda() for n in "qkv"), cu, softmax_type=st, window=90)
        bad.zero_()
        bad[2:, 150 + 133:150 + 133 + 91] = True
        _clean()
        assert torch.equal(torch.isnan(lse), bad) and torch.isnan(o[283:374, 2:]).all()
        assert torch.equal(lse[~bad], base[1][~bad])


def _fill_cache(k, v, lens, page):
    """The packed keys and values in a new 4-bit cache: pool, page table."""
    sdpa = _sdpa()
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    pool = sdpa.kv4_pool(at, k.shape[1], k.shape[2], page)
    sdpa.attn_kv4_append(k, v, _cu(lens), pool, table.cuda(), _i32([0] * len(lens)))
    return pool, table.cuda()


def _probabilities(q, k, keys):
    """fp64 softmax of q [n, H, d] over k [m, H_kv, d], row i over the first keys[i] keys; [H, n, m]."""
    q, k = q.double().cpu().numpy(), k.double().cpu().numpy()
    G = q.shape[1] // k.shape[1]
    s = np.stack([q[:, h] @ k[:, h // G].T for h in range(q.shape[1])]) / np.sqrt(q.shape[2])
    s = np.where(np.arange(k.shape[0]) < np.asarray(keys)[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


def test_newest_token_over_the_cache_and_over_the_gathered_cache():
    """Attention of the newest tokens over the cache, and packed attention of the same tokens over the
    cache read back.  Each rounds P and o to bf16, 2^-8 each; a score is an fp32 sum of 128 products, off by
    at most 2^-17 scale sum_x |q_x k_x|, 2^-13 for sums up to 16, and P by twice that, exponentials and
    sums included: 2^-11.  So |error| <= 2^-8 (sum_j P_j |v_j| + |o|) + 2^-11 sum_j P_j |v_j|, and the two
    differ by at most twice that."""
    sdpa = _sdpa()
    lens, H, H_kv, d, page = [300, 17, 129], 8, 2, 128, 32
    x = _inputs(lens, lens, H, H_kv, d, d, 31)
    q, k, v = (x[n].cuda() for n in "qkv")
    pool, table = _fill_cache(k, v, lens, page)
    last = torch.tensor(np.cumsum(lens) - 1, device="cuda")
    o, lse = sdpa.sdpa_decode_kv4(q[last].unsqueeze(1).contiguous(), pool, table, _i32(lens))
    kc, vc = sdpa.kv4_gather(pool, table, _cu(lens), _i32([0, 0, 0]), sum(lens), d)
    o2, lse2 = sdpa.sdpa_forward_packed(q[last].contiguous(), kc, vc, _cu([1, 1, 1]), _cu(lens), causal=False)
    _clean()
    at = np.cumsum([0] + lens)
    for b, n in enumerate(lens):
        sl = slice(int(at[b]), int(at[b + 1]))
        p = _probabilities(q[last[b]][None], kc[sl], [n])[:, 0]
        vv = vc[sl].double().cpu().numpy().repeat(H // H_kv, 1)
        exact, mag = np.einsum("hj,jhx->hx", p, vv), np.einsum("hj,jhx->hx", p, np.abs(vv))
        bound = 2.0 ** -8 * (mag + np.abs(exact)) + 2.0 ** -11 * mag
        one, two = o[b, 0].double().cpu().numpy(), o2[b].double().cpu().numpy()
        assert np.all(np.abs(one - exact) <= bound) and np.all(np.abs(two - exact) <= bound)
        assert np.all(np.abs(one - two) <= 2 * bound)
    assert (lse[:, :, 0].t() - lse2).abs().max() <= TOL_LSE


def test_prefill_of_several_tokens_over_a_cached_prefix():
    """A continuation's rows attend over the cached prefix, read back, without a causal mask and over their
    own rows with one; the two results joined by their lse are the attention over both.  Each result is
    within 2^-8 (sum_j P_j |v_j| + |o|) + 2^-11 sum_j P_j |v_j| of its own value (P over its own keys, the
    terms as in the test above), and |o| <= sum_j P_j |v_j|: with exact weights w and 1 - w the join is
    within (2^-7 + 2^-11) sum_j P_j |v_j|, P over all keys.  Each lse is off by at most 2^-12, so w by at
    most w (1 - w) 2^-11: another 2^-11 of that sum."""
    sdpa = _sdpa()
    H, H_kv, d, page = 8, 2, 128, 32
    prefix, new = [300, 17, 129, 64], [5, 200, 1, 130]
    xp, xn = _inputs(prefix, prefix, H, H_kv, d, d, 55), _inputs(new, new, H, H_kv, d, d, 56)
    pool, table = _fill_cache(xp["k"].cuda(), xp["v"].cuda(), prefix, page)
    kp, vp = sdpa.kv4_gather(pool, table, _cu(prefix), _i32([0] * 4), sum(prefix), d)
    q, k, v = (xn[n].cuda() for n in "qkv")
    o1, l1 = sdpa.sdpa_forward_packed(q, kp, vp, _cu(new), _cu(prefix), causal=False)
    o2, l2 = sdpa.sdpa_forward_packed(q, k, v, _cu(new))
    w = torch.sigmoid(l1 - l2).t()[..., None]
    o = (w * o1.float() + (1 - w) * o2.float()).double().cpu().numpy()
    lse = torch.logaddexp(l1, l2)
    _clean()
    ap, an = np.cumsum([0] + prefix), np.cumsum([0] + new)
    for b, (m, n) in enumerate(zip(prefix, new)):
        sp, sn = slice(int(ap[b]), int(ap[b + 1])), slice(int(an[b]), int(an[b + 1]))
        kk, vv = (torch.cat([a[sp], c[sn]]) for a, c in ((kp, k), (vp, v)))
        p = _probabilities(q[sn], kk, m + 1 + np.arange(n))
        vv = vv.double().cpu().numpy().repeat(H // H_kv, 1)
        exact, mag = np.einsum("hij,jhx->ihx", p, vv), np.einsum("hij,jhx->ihx", p, np.abs(vv))
        assert np.all(np.abs(o[sn] - exact) <= (2.0 ** -7 + 2.0 ** -10) * mag), f"sequence {b}"
        kd = kk.double().cpu().numpy().repeat(H // H_kv, 1)
        s = np.einsum("ihx,jhx->hij", q[sn].double().cpu().numpy(), kd) / np.sqrt(d)
        s = np.where(np.arange(m + n) < (m + 1 + np.arange(n))[:, None], s, -np.inf)
        ref = s.max(-1) + np.log(np.exp(s - s.max(-1, keepdims=True)).sum(-1))
        assert np.abs(lse[:, sn].double().cpu().numpy() - ref).max() <= TOL_LSE
