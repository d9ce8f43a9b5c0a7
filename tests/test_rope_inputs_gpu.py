"""Rotations whose inputs are written by the kernel right before them on the stream.

The rotation and the append with rotation are set up while that kernel still runs, so nothing they read may
be taken from before its end: a table buffer is written for one set of positions after another, keys and values
come from a rotation in place, offsets, lengths and page tables from copies, each followed by its reader at once.
Every result is compared bit for bit with the same calls waited for one by one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

STEPS = 12


def _sdpa():
    import scaled_dot_product_tmem_gb300 as sdpa
    return sdpa


def _clean():
    torch.cuda.synchronize()
    st, site = _sdpa().attn_last_device_error()
    assert st == 0, f"device error status {st} site {site:#x}"


def _randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [3, 700, 5001])
@pytest.mark.parametrize("d,rot,first,il", [(64, 64, 0, False), (128, 128, 0, False), (128, 64, 8, True), (64, 32, 16, True)])
def test_one_table_buffer_for_positions_one_after_another(d, rot, first, il, T, captured):
    sdpa = _sdpa()
    H, Hk, page = 4, 2, 32
    kw = dict(interleaved=il, first_dim=first)
    q, k, v = _randn(T, H, d, seed=1), _randn(T, Hk, d, seed=2), _randn(T, Hk, d, seed=3)
    inv, gain = sdpa.rope_frequencies(rot)
    pos = [torch.arange(T, dtype=torch.int32, device="cuda") * (i + 1) + 1009 * i for i in range(STEPS)]
    n_pages = -(-T // page)
    pages = torch.randperm(n_pages, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(1, -1).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros((T, 2, rot // 2), device="cuda")

    def steps(wait):
        out = []
        for i, p in enumerate(pos):
            pool = sdpa.kv4_pool(n_pages, Hk, d, page).zero_()
            sdpa.attn_rope_table(inv, p, table, gain=gain)
            wait()
            if i % 2:
                out += [*sdpa.rope_forward(q, k, table, **kw)]
            else:
                out += [sdpa.kv4_append_rope(q, k, v, table, cu, pool, pages, start, **kw), pool]
            wait()
        return out

    want = steps(torch.cuda.synchronize)
    if captured:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got = steps(lambda: None)
        g.replay()
    else:
        got = steps(lambda: None)
    _clean()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_offsets_and_pages_written_right_before_the_append(d, il):
    """Keys and values are the results of a rotation in place, which is itself set up early; then the offsets, the
    lengths and the page table are copied into their buffers before the next append."""
    sdpa = _sdpa()
    H, Hk, page, T = 4, 3, 16, 900
    inv, _ = sdpa.rope_frequencies(d)
    table = sdpa.rope_table(inv, torch.arange(T, dtype=torch.int32, device="cuda"))
    cuts = [[0, 1, T], [0, 500, T], [0, T - 1, T], [0, 0, T]]
    n_pages = 2 * (T // page + 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu, start = i32([0, 0, 0]), i32([0, 0])
    pages = torch.full((2, T // page + 2), -1, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(5)
    tables = [torch.randperm(n_pages, generator=gen).to(torch.int32).view(2, -1).cuda() for _ in cuts]
    cus, starts = [i32(c) for c in cuts], [i32([i, 2 * i + 1]) for i in range(len(cuts))]

    def steps(wait):
        q, k, v = _randn(T, H, d, seed=6), _randn(T, Hk, d, seed=7), _randn(T, Hk, d, seed=8)
        out = []
        for i in range(len(cuts)):
            pool = sdpa.kv4_pool(n_pages, Hk, d, page).zero_()
            cu.copy_(cus[i])
            start.copy_(starts[i])
            pages.copy_(tables[i])
            wait()
            sdpa.attn_rope(k, v, table, k, v, interleaved=il)
            wait()
            out += [sdpa.kv4_append_rope(q, k, v, table, cu, pool, pages, start, interleaved=il), pool, k.clone()]
            wait()
            pages.copy_(tables[i - 1])
            pool = sdpa.kv4_pool(n_pages, Hk, d, page).zero_()
            start.copy_(starts[i - 1])
            wait()
            out += [sdpa.kv4_append_rope(q, k, v, table, cu, pool, pages, start, interleaved=il), pool]
            wait()
        return out

    want = steps(torch.cuda.synchronize)
    for _ in range(3):
        got = steps(lambda: None)
        _clean()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("gain", [1.0, 1.375])
@pytest.mark.parametrize("sign", [1, -1])
def test_table_of_slow_and_negative_frequencies(sign, gain):
    """Against extended precision, up to the last int32 position, within what the number format leaves.

    A frequency becomes f turns a position with two roundings of 2^-53 (of 1 / 2 pi and of the product), held as a
    multiple of 2^-64: an angle is off by at most |p| (2^-64 + 2^-52 f) turns.  What is left after quarter turns is at most
    pi / 4 in fp32, off by 3 roundings (2.4 of 2^-24); sine and cosine turn that into at most 2.4 and 2 of 2^-24,
    their series and its roundings add at most 1.1 and 2.1 of 2^-24, the product with the gain one: 6 of 2^-24 in all."""
    from oracle import tree
    sdpa = _sdpa()
    gen = torch.Generator().manual_seed(9)
    w = torch.cat([10.0 ** -(torch.rand(96, generator=gen, dtype=torch.float64) * 12),
                   torch.tensor([1e-300, 2.0 ** -66, 1.0, 6.0, 7.0, 100.5, 1e-9, 0.0], dtype=torch.float64)]) * sign
    pos = torch.cat([torch.tensor([0, 1, -1, 131071, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64),
                     torch.randint(-2 ** 31, 2 ** 31, (200,), generator=gen)]).to(torch.int32)
    got = sdpa.rope_table(w.cuda(), pos.cuda(), gain=gain).double().cpu()
    a = torch.from_numpy(tree.angles(pos.numpy(), w.numpy()))
    turns = pos.double().abs()[:, None] * (2.0 ** -64 + 2.0 ** -52 * w.abs()[None] / (2 * torch.pi))
    bound = gain * (6 * 2.0 ** -24 + 2 * torch.pi * turns)
    for y, ref in ((got[:, 0], a.cos()), (got[:, 1], a.sin())):
        assert bool(((y - gain * ref).abs() <= bound).all()), float(((y - gain * ref).abs() - bound).max())
    _clean()


def test_a_gradient_whose_table_was_rewritten_is_refused():
    """Two micro-batches whose tables share a buffer: the first one's gradient must not turn by the second's angles."""
    sdpa = _sdpa()
    T, H, d = 5, 2, 64
    inv, _ = sdpa.rope_frequencies(d)
    q = _randn(T, H, d, seed=1).requires_grad_()
    table = torch.empty((T, 2, d // 2), device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    for other_stream in (False, True):
        sdpa.attn_rope_table(inv, pos, table)
        y, _ = sdpa.rope(q, None, table)
        s = torch.cuda.Stream() if other_stream else None
        torch.cuda.synchronize()
        sdpa.attn_rope_table(inv, pos + 100, table, stream=s)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward(torch.ones_like(y))
    assert q.grad is None
    with torch.inference_mode():  # tensors without a version
        t = torch.empty((T, 2, d // 2), device="cuda")
        sdpa.attn_rope_table(inv, pos, t)
        sdpa.attn_rope(q, None, t, torch.empty_like(q), None)
    _clean()


def test_rotation_in_place_within_a_graph_is_refused():
    sdpa = _sdpa()
    T, H, d = 96, 2, 64
    inv, _ = sdpa.rope_frequencies(d)
    table = sdpa.rope_table(inv, torch.arange(T, dtype=torch.int32, device="cuda"))
    x = _randn(T, H, d, seed=1).requires_grad_()
    y = x * 2
    held = y.detach().clone()
    with pytest.raises(ValueError, match="differentiable"):
        sdpa.attn_rope(y, None, table, y, None)
    with pytest.raises(ValueError, match="differentiable"):
        sdpa.attn_rope(x.detach(), x.detach(), table, torch.empty_like(held), y)
    assert torch.equal(y.detach(), held)
    # queries that attention keeps for its gradient, turned afterwards
    q, k, v = (_randn(1, T, H, d, seed=s) for s in (2, 3, 4))
    v.requires_grad_()
    o = sdpa.attention(q, k, v)
    sdpa.attn_rope(q, None, table, q, None)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.backward(torch.ones_like(o))
    with torch.no_grad():
        sdpa.attn_rope(y, None, table, y, None)
        assert torch.equal(y, sdpa.rope_forward(held, None, table)[0])
    _clean()
