"""Rotary positions on the GPU: the table against extended precision, rotations bit for bit against the
same roundings in torch, gradients, strided and in-place rows, and keys rotated on their way into the
4-bit cache.

Bounds.  A table entry: the angle is reduced to its nearest quarter turn in whole-number arithmetic, off only by the
frequency's two roundings and its last bit (the test's own term for far positions).  What is left, at most pi / 4, takes
three roundings to fp32 (2.4 of 2^-24); sine and cosine, power series to x^9 and x^8 whose left-out terms are below 2^-29
and 2^-25, turn that and their own roundings into at most 4.2 of 2^-24, the gain's product adds one: within 2^-21 gain
in all.  A rotated value is
two products, a sum and a rounding to bf16: 2^-8 |y| + 2^-22 (|x1 c| + |x2 s|)."""
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


def _randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _rounded(x, table, first, interleaved, inverse=False):
    """The rotation in torch with the documented roundings: x [T, H, d] bf16 and table [T, 2, n] on the CPU."""
    n = table.shape[2]
    c, s = table[:, None, 0], table[:, None, 1]
    if inverse:
        s = -s
    i1, i2 = (torch.from_numpy(i) for i in tree.pairs(n, first, interleaved))
    f = x.float()
    y = f.clone()
    y[..., i1] = f[..., i1] * c - f[..., i2] * s
    y[..., i2] = f[..., i2] * c + f[..., i1] * s
    return y.to(torch.bfloat16)


@pytest.mark.parametrize("n,base,gain", [(64, 10000.0, 1.0), (32, 500000.0, 1.25), (8, 100.0, 0.5), (128, 1e6, 1.0),
                                         (24, 10000.0, 1.0)])
def test_table_at_near_and_far_positions(n, base, gain):
    sdpa = _sdpa()
    inv, _ = sdpa.rope_frequencies(2 * n, base=base)
    pos = [0, 1, 2, 3, 1000, 4095, 131071, 999999, 2 ** 24 + 1, 2 ** 31 - 1, -1, -12345, -2 ** 31]
    pos += np.random.default_rng(n).integers(0, 2 ** 20, 300).tolist()
    t = sdpa.rope_table(inv, _i32(pos), gain=gain).double().cpu().numpy()
    a = tree.angles(pos, inv.cpu().numpy())
    # (the frequency itself, in turns, is off by 2^-52 of it: up to 2^31 2^-52 2 pi radians here)
    far = np.abs(np.asarray(pos, np.float64))[:, None] * inv.cpu().numpy()[None] * 2.0 ** -51
    for got, ref in ((t[:, 0], np.cos(a)), (t[:, 1], np.sin(a))):
        assert np.all(np.abs(got - gain * ref) <= gain * (2.0 ** -21 + far))
    _clean()


def test_table_shapes():
    sdpa = _sdpa()
    inv, _ = sdpa.rope_frequencies(32)
    assert sdpa.rope_table(inv, _i32([])).shape == (0, 2, 16)
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    assert torch.equal(sdpa.rope_table(inv, pos), sdpa.rope_table(inv, pos.view(-1)))


CASES = [  # T, H, H_k, d, n, first, interleaved
    (1, 1, 1, 16, 8, 0, False),
    (7, 3, 1, 64, 32, 0, False),
    (5, 8, 2, 128, 64, 0, True),
    (130, 4, 4, 192, 32, 128, False),
    (33, 2, 0, 96, 24, 16, True),
    (9, 5, 3, 64, 8, 8, False),
    (21, 7, 7, 40, 16, 0, True),      # one dim block of 8 stays behind the pairs
    (4, 2, 1, 256, 128, 0, False),
    (600, 33, 9, 128, 32, 40, False),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,H_k,d,n,first,il", CASES)
def test_rotation_bits_and_bound(T, H, H_k, d, n, first, il, inverse):
    sdpa = _sdpa()
    q, k = _randn(T, H, d, seed=1), _randn(T, H_k, d, seed=2) if H_k else None
    inv, _ = sdpa.rope_frequencies(2 * n)
    table = sdpa.rope_table(inv, _i32(list(range(3, T + 3))), gain=1.125)
    fn = sdpa.rope_backward if inverse else sdpa.rope_forward
    out = fn(q.cuda(), None if k is None else k.cuda(), table, interleaved=il, first_dim=first)
    _clean()
    tc = table.cpu()
    for x, y in zip((q, k), out):
        if x is None:
            assert y is None
            continue
        assert torch.equal(y.cpu(), _rounded(x, tc, first, il, inverse))
        c, s = tc[:, 0].double().numpy(), tc[:, 1].double().numpy()
        xd = x.double().numpy()
        ref = tree.rotate(xd, c, -s if inverse else s, first, il)
        # |x1 c| + |x2 s| of both values of a pair
        mag = np.maximum(*(tree.rotate(np.abs(xd), np.abs(c), sign * np.abs(s), first, il) for sign in (1, -1)))
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * mag)


def test_strided_in_place_and_shared_positions():
    """Slices of a fused projection, in place and out of it; a batch that shares its positions."""
    sdpa = _sdpa()
    B, S, H, Hk, d = 3, 17, 4, 2, 64
    fused = _randn(B, S, (H + 2 * Hk) * d, seed=3).cuda()
    before = fused.clone()
    inv, _ = sdpa.rope_frequencies(32)
    table = sdpa.rope_table(inv, _i32(list(range(100, 100 + S))))
    cut = lambda t: (t[..., :H * d].unflatten(-1, (H, d)), t[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d)))
    q, k = cut(fused)
    q2, k2 = sdpa.rope_forward(q, k, table, first_dim=16)
    full = table.repeat(B, 1, 1)
    q3, k3 = sdpa.rope_forward(q.reshape(B * S, H, d), k.reshape(B * S, Hk, d), full, first_dim=16)
    assert torch.equal(q2.view(-1, H, d), q3) and torch.equal(k2.view(-1, Hk, d), k3)
    sdpa.attn_rope(q, k, table, q, k, first_dim=16)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(fused[..., (H + Hk) * d:], before[..., (H + Hk) * d:])
    assert torch.equal(cut(fused)[0][..., :16], cut(before)[0][..., :16])
    _clean()


def test_special_values_stay_in_their_pairs():
    sdpa = _sdpa()
    q = _randn(2, 1, 64, seed=4)
    q[0, 0, 3], q[1, 0, 40] = float("inf"), float("nan")
    inv, _ = sdpa.rope_frequencies(64)
    y = sdpa.rope_forward(q.cuda(), None, sdpa.rope_table(inv, _i32([5, 6])))[0].float().cpu()
    bad = ~torch.isfinite(y)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 35] and bad[1, 0].nonzero().flatten().tolist() == [8, 40]


@pytest.mark.parametrize("il", [False, True])
def test_gradient_against_formula_and_differences(il):
    """The rotation is linear: <rope(x + u) - rope(x - u), g> / 2 = <u, gradient>, within the roundings of
    both sides; and the gradient is the transposed rotation, bit for bit."""
    sdpa = _sdpa()
    T, H, Hk, d, n = 11, 3, 2, 64, 16
    q, k = _randn(T, H, d, seed=5).cuda().requires_grad_(), _randn(T, Hk, d, seed=6).cuda().requires_grad_()
    inv, _ = sdpa.rope_frequencies(2 * n)
    table = sdpa.rope_table(inv, _i32(list(range(T))), gain=1.1)
    y, z = sdpa.rope(q, k, table, interleaved=il, first_dim=8)
    gq, gk = _randn(T, H, d, seed=7).cuda(), _randn(T, Hk, d, seed=8).cuda()
    torch.autograd.backward([y, z], [gq, gk])
    assert torch.equal(q.grad.cpu(), _rounded(gq.cpu(), table.cpu(), 8, il, True))
    assert torch.equal(k.grad.cpu(), _rounded(gk.cpu(), table.cpu(), 8, il, True))
    u = _randn(T, H, d, seed=9).cuda()
    with torch.no_grad():
        up = sdpa.rope_forward(q.detach() + u, None, table, interleaved=il, first_dim=8)[0].double()
        dn = sdpa.rope_forward(q.detach() - u, None, table, interleaved=il, first_dim=8)[0].double()
    # the points themselves are bf16: use their true distance
    du = ((q.detach() + u).double() - (q.detach() - u).double()) / 2
    lhs = ((up - dn) / 2 * gq.double()).sum()
    rhs = (du * q.grad.double()).sum()
    bound = 2.0 ** -8 * (((up.abs() + dn.abs()) / 2 * gq.double().abs()).sum() + (du.abs() * q.grad.double().abs()).sum())
    assert abs(float(lhs - rhs)) <= float(bound)


def test_gradients_of_one_output_and_uneven_rows():
    sdpa = _sdpa()
    T, H, Hk, d = 6, 2, 1, 32
    q, k = _randn(T, H, d, seed=1).cuda().requires_grad_(), _randn(T, Hk, d, seed=2).cuda().requires_grad_()
    inv, _ = sdpa.rope_frequencies(32)
    table = sdpa.rope_table(inv, _i32(list(range(T))))
    y, z = sdpa.rope(q, k, table)
    z.float().sum().backward()            # an expanded gradient, and none for q
    assert q.grad is None
    ones = torch.ones((T, Hk, d), dtype=torch.bfloat16)
    assert torch.equal(k.grad.cpu(), _rounded(ones, table.cpu(), 0, False, True))
    k.grad = None
    y, _ = sdpa.rope(q, None, table)
    (y.transpose(0, 1).contiguous().float() ** 2).sum().backward()
    assert q.grad is not None and k.grad is None


@pytest.mark.parametrize("packed", [False, True])
def test_attention_with_rotation_equals_its_parts(packed):
    sdpa = _sdpa()
    B, S, H, Hk, d = 2, 96, 4, 2, 64
    inv, gain = sdpa.rope_frequencies(d, scaling="parts", factor=4.0, original_length=64)
    table = sdpa.rope_table(inv, _i32(list(range(S))), gain=gain)
    mk = lambda h, s: _randn(B, S, h, d, seed=s).cuda()
    grads = []
    for fused in (False, True):
        q, k, v = (t.requires_grad_() for t in (mk(H, 1), mk(Hk, 2), mk(Hk, 3)))
        if packed:
            cu, t2 = _i32([0, S, 2 * S]), table.repeat(B, 1, 1)
            a, b, c = (t.reshape(B * S, -1, d) for t in (q, k, v))
            if fused:
                o = sdpa.attention_packed(a, b, c, cu, rope=t2)
            else:
                o = sdpa.attention_packed(*sdpa.rope(a, b, t2), c, cu)
            o = o.view(B, S, H, d)
        elif fused:
            o = sdpa.attention(q, k, v, rope=table)
        else:
            o = sdpa.attention(*sdpa.rope(q, k, table), v)
        o.backward(mk(H, 4))
        grads.append([o.detach(), q.grad, k.grad, v.grad])
    for a, b in zip(*grads):
        assert torch.equal(a, b)
    # and the rotated heads' attention is a function of distances: shifted positions change nothing but roundings
    q, k, v = mk(H, 1), mk(Hk, 2), mk(Hk, 3)
    o0 = sdpa.attention(q, k, v, rope=sdpa.rope_table(inv, _i32(list(range(S)))))
    o1 = sdpa.attention(q, k, v, rope=sdpa.rope_table(inv, _i32(list(range(7000, 7000 + S)))))
    rel = float((o0.float() - o1.float()).norm() / o0.float().norm())
    assert rel <= 2.0 ** -5  # bf16 roundings of q, k (2^-8 each of scores of a few units), of P and of o
    _clean()


# ------------------------------------------------------------------------------------------ into the cache


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("d,n,first,il", [(64, 32, 0, False), (64, 16, 8, True), (128, 64, 0, False), (128, 24, 8, False),
                                          (128, 64, 0, True), (128, 8, 112, False)])
def test_append_rotated_is_rotation_then_append(page, d, n, first, il):
    """Cache bytes and queries are those of the separate calls; other bytes stay; k and v as slices."""
    sdpa = _sdpa()
    lens, start, Hk, H = [5, 0, 33, 1, 70], [3, 0, 14, 0, 60], 3, 6
    T = sum(lens) + 4  # four rows of no sequence
    fused = _randn(T, (H + 2 * Hk) * d, seed=page + n).cuda()
    q, k, v = (t.unflatten(-1, (-1, d)) for t in fused.split([H * d, Hk * d, Hk * d], -1))
    need = [-(-(a + b) // page) for a, b in zip(lens, start)]
    n_pages = sum(need)
    table = torch.full((5, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.arange(at, at + m, dtype=torch.int32)
        at += m
    table = table.cuda()
    cu = _i32([0] + np.cumsum(lens).tolist())
    inv, _ = sdpa.rope_frequencies(2 * n)
    rt = sdpa.rope_table(inv, torch.arange(T, dtype=torch.int32, device="cuda") * 3)
    pools = [torch.full((n_pages, Hk, sdpa.kv4_block_bytes(page, d)), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(3)]
    qr, kr = sdpa.rope_forward(q, k, rt, interleaved=il, first_dim=first)
    sdpa.attn_kv4_append(kr, v, cu, pools[0], table, _i32(start))
    got = sdpa.kv4_append_rope(q, k, v, rt, cu, pools[1], table, _i32(start), interleaved=il, first_dim=first)
    assert torch.equal(got, qr) and torch.equal(pools[0], pools[1])
    assert sdpa.kv4_append_rope(None, k, v, rt, cu, pools[2], table, _i32(start), interleaved=il, first_dim=first) is None
    assert torch.equal(pools[0], pools[2])
    _clean()


def test_append_rotated_values_against_the_oracle():
    """Held keys are the format's values of the rotated keys (bf16), for 3 tokens at far positions."""
    sdpa = _sdpa()
    d, page, Hk = 128, 16, 2
    k, v = _randn(3, Hk, d, seed=1), _randn(3, Hk, d, seed=2)
    inv, _ = sdpa.rope_frequencies(d)
    rt = sdpa.rope_table(inv, _i32([100000, 100001, 7]))
    pool = sdpa.kv4_pool(1, Hk, d, page)
    sdpa.kv4_append_rope(None, k.cuda(), v.cuda(), rt, _i32([0, 3]), pool, _i32([[0]]), _i32([4]))
    gk, gv = sdpa.kv4_gather(pool, _i32([[0]]), _i32([0, 3]), _i32([4]), 3, d)
    kr = _rounded(k, rt.cpu(), 0, False).double().numpy()
    assert np.array_equal(gk.double().cpu().numpy(), kv4.held(kr))
    assert np.array_equal(gv.double().cpu().numpy(), kv4.held(v.double().numpy()))


def test_captured_and_on_another_stream():
    sdpa = _sdpa()
    q, k = _randn(40, 4, 64, seed=1).cuda(), _randn(40, 2, 64, seed=2).cuda()
    inv, _ = sdpa.rope_frequencies(64)
    pos = _i32(list(range(40)))
    ref = sdpa.rope_forward(q, k, sdpa.rope_table(inv, pos))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sdpa.rope_forward(q, k, sdpa.rope_table(inv, pos, stream=s), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = sdpa.rope_forward(q, k, sdpa.rope_table(inv, pos))
    pos.add_(5)
    want = sdpa.rope_forward(q, k, sdpa.rope_table(inv, pos))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "join of streams", "another operator"])
def test_captured_behind(before):
    """Rotation and append with rotation as a graph's first node, behind a copy, a fill, two streams, attention."""
    sdpa = _sdpa()
    T, H, Hk, d = 48, 4, 2, 64
    x, k = _randn(T, H, d, seed=1).cuda(), _randn(T, Hk, d, seed=2).cuda()
    q = torch.zeros_like(x)
    inv, _ = sdpa.rope_frequencies(d)
    table = sdpa.rope_table(inv, _i32(list(range(T))))
    pages, cu, start = _i32([[0, 1, 2, 3]]), _i32([0, T]), _i32([0])
    pool = sdpa.kv4_pool(4, Hk, d, 16)
    side = torch.cuda.Stream()
    o = torch.empty_like(x)

    def step():
        if before == "copy":
            q.copy_(x)
        elif before == "fill":
            q.zero_()
            q.add_(x)
        elif before == "join of streams":
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                q.copy_(x)
            o.copy_(x)
            main.wait_stream(side)
        elif before == "another operator":
            q.copy_(sdpa.sdpa_forward_packed(x, k, k, cu)[0])
        a = sdpa.rope_forward(q, k, table)
        return (*a, sdpa.kv4_append_rope(q, k, k, table, cu, pool, pages, start))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (5, 6):
        x.copy_(_randn(T, H, d, seed=seed).cuda())
        if before == "nothing":
            q.copy_(x)
        pool.zero_()
        g.replay()
        torch.cuda.synchronize()
        held = pool.clone()
        pool.zero_()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        assert torch.equal(pool, held)
    _clean()


def test_gradient_of_the_gradient():
    """The rotation is linear: the gradient of <rotated back w, u> by w is u rotated."""
    sdpa = _sdpa()
    inv, gain = sdpa.rope_frequencies(32)
    table = sdpa.rope_table(inv, _i32([5, 0, 77]))
    q, k = (_randn(3, h, 64, seed=h).cuda().requires_grad_() for h in (4, 2))
    wq, wk = (_randn(3, h, 64, seed=10 + h).cuda().requires_grad_() for h in (4, 2))
    uq, uk = (_randn(3, h, 64, seed=20 + h).cuda() for h in (4, 2))
    grads = torch.autograd.grad(sdpa.rope(q, k, table, first_dim=16), (q, k), (wq, wk), create_graph=True)
    for got, want in zip(grads, sdpa.rope_backward(wq.detach(), wk.detach(), table, first_dim=16)):
        assert torch.equal(got, want)
    second = torch.autograd.grad(grads, (wq, wk), (uq, uk))
    for got, want in zip(second, sdpa.rope_forward(uq, uk, table, first_dim=16)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("packed", [False, True])
def test_training_step_captured(packed):
    """Attention with positions, forward and backward, replayed with other inputs."""
    sdpa = _sdpa()
    B, S, H, d = 2, 96, 2, 64
    shape = (B * S, H, d) if packed else (B, S, H, d)
    q, k, v, w = (_randn(*shape, seed=i).cuda() for i in range(4))
    for t in (q, k, v):
        t.requires_grad_()
    inv, _ = sdpa.rope_frequencies(d)
    pos, cu = torch.arange(S, dtype=torch.int32, device="cuda"), _i32([0, S, 2 * S])

    def step():
        table = sdpa.rope_table(inv, pos.repeat(B) if packed else pos)
        if packed:
            o = sdpa.attention_packed(q, k, v, cu, rope=table)
        else:
            o = sdpa.attention(q, k, v, rope=table)
        return (o.detach(), *torch.autograd.grad(o, (q, k, v), w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    with torch.no_grad():
        q.copy_(_randn(*shape, seed=9).cuda())
        pos.add_(1000)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    _clean()


def test_python_refusals():
    sdpa = _sdpa()
    inv, _ = sdpa.rope_frequencies(32)
    table = sdpa.rope_table(inv, _i32([0, 1, 2, 3]))
    q, k = _randn(4, 2, 64).cuda(), _randn(4, 1, 64).cuda()
    with pytest.raises(ValueError, match="one row per row"):
        sdpa.rope_forward(q[:2], k[:2], table)
    with pytest.raises(ValueError, match="shapes of q and k"):
        sdpa.attn_rope(q, k, table, torch.empty_like(q), None)
    with pytest.raises(ValueError, match="shapes of q and k"):
        sdpa.attn_rope(q, None, table, torch.empty_like(k), None)
    with pytest.raises(ValueError, match="q's rows"):
        sdpa.rope_forward(q, k[:3], table)
    with pytest.raises(TypeError):
        sdpa.rope_forward(q.half(), k.half(), table)
    with pytest.raises(TypeError):
        sdpa.rope_table(inv.float(), _i32([0]))
    with pytest.raises(TypeError):
        sdpa.rope_table(inv, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="evenly apart"):
        sdpa.rope_forward(_randn(2, 4, 4, 64).cuda()[:, :2], None, table)
    with pytest.raises(ValueError, match="contiguous"):
        sdpa.rope_forward(q.transpose(1, 2), None, table)
    with pytest.raises(sdpa.AttnError):
        sdpa.rope_forward(q, k, table, first_dim=40)     # past the head
    with pytest.raises(sdpa.AttnError):
        sdpa.rope_forward(q, k, table, first_dim=4)      # not a multiple of 8
    with pytest.raises(sdpa.AttnError):
        sdpa.rope_forward(_randn(4, 1, 264).cuda(), None, table)
    with pytest.raises(sdpa.AttnError):                    # rows start off a 16-byte boundary
        sdpa.rope_forward(_randn(4 * 2 * 64 + 4).cuda()[4:].view(4, 2, 64), None, table)
