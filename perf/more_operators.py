"""Cases of rotary positions and of speculative serving over the 4-bit paged key/value cache.

Four operators around fused attention:

  rope    cos/sin of the rows' positions, and queries and keys rotated by them; forward, or forward and
          backward
  append  keys rotated and quantised on their way into the 4-bit cache, values quantised, queries rotated;
          the new tokens read back
  tree    attention of a tree of drafted tokens over a sequence's 4-bit cache
  keep    after verification: the cache entries of the accepted nodes moved to the end of their sequence

`run` computes each either with elementary torch operations (`own` false) or through this package's
entry points (`own` true).  `exact` gives the same outputs from the definitions in 64 bits.

Rotation.  Dims first .. first + 2n of a head hold n pairs: (f, f + n) in the half layout, (2f, 2f + 1)
in the interleaved one.  A pair (x1, x2) becomes (x1 c - x2 s, x2 c + x1 s), c = gain cos(p w_f), s = gain sin(p w_f),
p the row's position.  The frequencies w_f are base^(-f/n), for long contexts scaled: "linear" (divided by
the factor), "base" (the base times factor^(n/(n-1))) or "parts" (pairs that turn less than once in the
original length are divided by the factor, pairs that turn 32 times or more are kept, those between are
blended; the gain is 0.1 ln(factor) + 1).

The tree.  The nodes of sequence b are its tokens L, L + 1, ... in the cache; node i's position is L plus
its depth.  It sees the L tokens before the tree, its ancestors and itself, under a window of w only
positions of at least its own minus w.

The cache.  A pool holds pages [n_pages, H_kv, block]; the block of one page and one head holds
P tokens of head dim d as four consecutive parts:
  K codes   [P][d/2]            two codes a byte, the even dim in the low nibble
  V codes   [P/2][8][2][d/16]   token pair u, eighth g of the head dim at slot g ^ x(u), the two tokens
  K scales  [P][d/16]           one byte for 16 dims
  V scales  [P/2][d/16][2]
with x(u) = 2 (u mod 4) at d = 128 and 4 (floor(u / 2) mod 2) at d = 64.  A code c in 0..15 stands
for (c - 8) s; a scale byte holds bits 14..7 of a half-precision number.  For 16 values x, s = max|x| / 7
rounded to that format (ties to even, at most 0xF7) and c = 8 + clamp(round(x / s), -8, 7).
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one new token for each of a few requests of a small model: what counts is the launch
        dict(name="rope_step_d64", op="rope", rows=8, S=0, far=900, H=8, H_kv=2, d=64, rot=64, first=0, interleaved=False,
             scaling="none", factor=1.0, train=False),
        # a batch of prompts of a model with its context extended, positions up to 131072
        dict(name="rope_prompts", op="rope", rows=32511, S=0, far=131072, H=32, H_kv=8, d=128, rot=128, first=0,
             interleaved=False, scaling="parts", factor=16.0, train=False),
        # a training step, half of each head rotated, pairs side by side
        dict(name="rope_train_half_head", op="rope", rows=16384, S=4096, far=0, H=32, H_kv=8, d=128, rot=64, first=0,
             interleaved=True, scaling="none", factor=1.0, train=True),
        # a training step with the rotated part behind the unrotated one (192 dims, the last 64 turn)
        dict(name="rope_train_tail", op="rope", rows=4099, S=0, far=5000, H=16, H_kv=16, d=192, rot=64, first=128,
             interleaved=False, scaling="linear", factor=4.0, train=True),
        # one token for each of many running requests enters the cache
        dict(name="append_step", op="append", lens=",".join(["1"] * 64), before="37", H=32, H_kv=8, d=128, rot=128, first=0,
             interleaved=False, page=16),
        # prompts enter the cache
        dict(name="append_prompts", op="append", lens="8192,4097,2000,1024,333,31", before="5", H=32, H_kv=8, d=128, rot=128,
             first=0, interleaved=False, page=64),
        # a small drafted tree of one request of a small model
        dict(name="tree_single_d64", op="tree", lens="200", nodes="7", chain=False, H=8, H_kv=2, d=64, page=16, window=-1,
             sink="vanilla"),
        # running requests of different age, trees of different sizes, a window and a learnable sink
        dict(name="tree_ragged_window", op="tree", lens="4096,1,777,8191,2500,64,65,3999,1200,5000,31,6144",
             nodes="1,24,13,32,9,60,5,27,16,3,40,31", chain=False, H=16, H_kv=4, d=64, page=32, window=2000, sink="learnable"),
        # a batch of running requests, 16 nodes each
        dict(name="tree_batch", op="tree", lens="4096,1,777,8191,2500,64,65,3999,1200,5000,31,6144,900,2047,16,7000",
             nodes=",".join(["16"] * 16), chain=False, H=32, H_kv=8, d=128, page=64, window=-1, sink="vanilla"),
        # long contexts, a large tree each
        dict(name="tree_long", op="tree", lens="131072,65536,100001,32768", nodes="64,64,61,64", chain=False, H=32, H_kv=8,
             d=128, page=64, window=-1, sink="vanilla"),
        # the accepted nodes of a few requests in one layer
        dict(name="keep_step", op="keep", B=16, most=5, nodes=16, before=100, layers=1, H_kv=8, d=128, page=16),
        # of many requests in all layers
        dict(name="keep_layers", op="keep", B=64, most=9, nodes=64, before=700, layers=32, H_kv=8, d=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, n_max, len_max, total_max):
    n = _log_int(rng, 1, n_max)
    top = _log_int(rng, 8, len_max)
    lens, total = [], 0
    for _ in range(n):
        v = rng.choice([_log_int(rng, 1, top), rng.randint(1, top)])
        v = min(v, total_max - total)
        if v <= 0:
            break
        lens.append(v)
        total += v
    return lens


def _text(numbers):
    return ",".join(map(str, numbers))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "keep"])
    H, H_kv = rng.choice([(32, 8), (8, 2), (16, 16), (32, 1), (24, 4), (64, 8), (7, 7)])
    if op == "rope":
        d, rot, first = rng.choice([(64, 64, 0), (128, 128, 0), (128, 64, 0), (128, 32, 0), (192, 64, 128), (96, 48, 0),
                                    (64, 16, 8), (256, 256, 0)])
        rows, S = _log_int(rng, 1, 12000), 0
        if rng.random() < 0.4:  # a padded batch: all entries have the same positions
            S = max(1, rows // rng.randint(1, 4))
            rows = rows // S * S
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return dict(op=op, rows=rows, S=S, far=_log_int(rng, 1, 1000000), H=H, H_kv=H_kv, d=d, rot=rot, first=first,
                    interleaved=rng.random() < 0.5, scaling=scaling, factor=rng.choice([2.0, 8.0, 40.0]),
                    train=rng.random() < 0.6)
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        rot = rng.choice([d, d, d // 2, 48])
        return dict(op=op, lens=_text(_draw_lens(rng, 64, 8000, 15000)), before=str(rng.randint(0, 300)), H=H, H_kv=H_kv, d=d,
                    rot=rot, first=rng.choice([0, 8]) if rot < d - 8 else 0, interleaved=rng.random() < 0.4, page=page)
    if op == "tree":
        lens = _draw_lens(rng, 32, 60000, 150000)
        top = _log_int(rng, 1, 64)
        lens = [0 if rng.random() < 0.05 else v for v in lens]
        return dict(op=op, lens=_text(lens), nodes=_text([rng.randint(1, top) for _ in lens]), chain=rng.random() < 0.3, H=H,
                    H_kv=H_kv, d=d, page=page, window=_log_int(rng, 1, 4096) if rng.random() < 0.3 else -1,
                    sink=rng.choice(["vanilla", "off_by_one", "learnable"]))
    nodes = _log_int(rng, 1, 64)
    return dict(op=op, B=_log_int(rng, 1, 64), most=rng.randint(1, min(nodes, 12)), nodes=nodes, before=rng.randint(0, 900),
                layers=rng.randint(1, 16), H_kv=H_kv, d=d, page=page)


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def work(case):
    op, d, H_kv = case["op"], case["d"], case["H_kv"]
    if op == "rope":
        table_rows = case["S"] or case["rows"]
        heads = case["rows"] * (case["H"] + H_kv)
        once = 2 * 2 * heads * d
        table = 4 * table_rows * case["rot"]
        n = 2 if case["train"] else 1
        return dict(bytes=n * once + table + 4 * table_rows, flops=n * 3 * heads * case["rot"])
    token = d * 9 // 8  # bytes of one token and head: codes and scales of K and V
    if op == "append":  # k, v and q read, q and the pages written, the pages read back
        T = sum(_ints(case["lens"]))
        return dict(bytes=T * (H_kv * (2 * 4 * d + 2 * token) + 2 * 2 * case["H"] * d + 4 * case["rot"]),
                    flops=T * (H_kv * 8 * d + 3 * case["H"] * case["rot"]))
    if op == "tree":
        lens, nodes, w = _ints(case["lens"]), _ints(case["nodes"]), case["window"]
        seen = [(min(L, w) if w >= 0 else L) for L in lens]
        rows = sum(nodes) * case["H"]
        pairs = sum((s + (n + 1) // 2) * n for s, n in zip(seen, nodes))
        return dict(bytes=sum(s + n for s, n in zip(seen, nodes)) * H_kv * token + rows * (4 * d + 4),
                    flops=4 * pairs * case["H"] * d)
    moved = case["B"] * (case["most"] + 1) // 2
    return dict(bytes=2 * moved * case["layers"] * H_kv * token + 4 * case["B"] * (case["most"] + 1), flops=0)


# ------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _kv_like(g, T, H, d, outlier):
    """Keys or values as projections make them; keys have a few large channels."""
    x = torch.randn((T, H, d), generator=g, device="cuda", dtype=torch.float32)
    if outlier:
        x[:, :, ::31] *= 6.0
    return x.to(torch.bfloat16)


def _table(g, need, n_pages):
    """Pages drawn without repetition: row b of the table lists need[b] of them, the rest is -1."""
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t


def _frequencies(rot, scaling="none", factor=1.0, base=10000.0, original=4096):
    """Radians a position of the rot / 2 pairs in 64 bits, and the gain."""
    n = rot // 2
    f = np.arange(n, dtype=np.float64) / n
    if scaling == "base":
        base *= factor ** (n / (n - 1))
    w = base ** -f
    if scaling == "linear":
        w = w / factor
    gain = 1.0
    if scaling == "parts":
        turns = original * w / (2 * math.pi)
        keep = np.clip((np.log(np.maximum(turns, 1e-300)) - 0.0) / math.log(32.0), 0.0, 1.0)
        w = w * keep + w / factor * (1 - keep)
        gain = 0.1 * math.log(factor) + 1.0
    return torch.from_numpy(w).cuda(), gain


def _parents(rng, nodes, chain):
    """Parents of every sequence's nodes, packed: -1 for a child of the last token before the tree."""
    out = []
    for n in nodes:
        out += [i - 1 if chain else int(rng.integers(max(-1, i - 7), i)) for i in range(n)]
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    rng = np.random.default_rng(seed)
    st = dict(case=case)
    H_kv, d = case["H_kv"], case["d"]
    if op == "rope":
        rows, H, S = case["rows"], case["H"], case["S"]
        st["inv_freq"], st["gain"] = _frequencies(case["rot"], case["scaling"], case["factor"])
        if S:
            st["positions"] = torch.arange(S, dtype=torch.int32, device="cuda") + case["far"]
        else:  # a few runs of consecutive positions, as packed sequences have
            at = torch.randint(0, max(1, case["far"] - rows // 4), (4,), generator=g, device="cuda")
            i = torch.arange(rows, device="cuda")
            st["positions"] = (at[i * 4 // rows] + i % ((rows + 3) // 4)).to(torch.int32)
        shape = (rows // S, S) if S else (rows,)
        fused = _randn(g, *shape, (H + 2 * H_kv) * d)  # one projection: q, k and v side by side
        st["q"] = fused[..., :H * d].unflatten(-1, (H, d))
        st["k"] = fused[..., H * d:(H + H_kv) * d].unflatten(-1, (H_kv, d))
        if case["train"]:
            st["dq"], st["dk"] = _randn(g, *shape, H, d), _randn(g, *shape, H_kv, d)
        return st
    P = case["page"]
    block = P * d * 9 // 8
    if op == "append":
        lens, before = _ints(case["lens"]), int(case["before"])
        need = [(before + n + P - 1) // P for n in lens]
        n_pages = sum(need) + 3
        w, gain = _frequencies(case["rot"])
        # cos and sin of the rows, made once for all layers of a step
        pos = torch.cat([torch.arange(before, before + n, device="cuda", dtype=torch.float64) for n in lens])
        a = pos[:, None] * w
        st.update(lens=lens, before=before, q=_randn(g, sum(lens), case["H"], d), k=_kv_like(g, sum(lens), H_kv, d, True),
                  v=_kv_like(g, sum(lens), H_kv, d, False), cu=_cu(lens), table=_table(g, need, n_pages),
                  rope=torch.stack([a.cos(), a.sin()], 1).float(),
                  starts=torch.full((len(lens),), before, dtype=torch.int32, device="cuda"),
                  pool=torch.randint(0, 256, (n_pages, H_kv, block), generator=g, device="cuda", dtype=torch.uint8))
        return st
    if op == "tree":
        lens, nodes = _ints(case["lens"]), _ints(case["nodes"])
        need = [(L + n + P - 1) // P for L, n in zip(lens, nodes)]
        n_pages = sum(need) + 1
        pool = torch.randint(0, 256, (n_pages, H_kv, block), generator=g, device="cuda", dtype=torch.uint8)
        table = _table(g, need, n_pages)
        for b, (L, n) in enumerate(zip(lens, nodes)):
            _write(pool, table[b], 0, _kv_like(g, L + n, H_kv, d, True), _kv_like(g, L + n, H_kv, d, False), P)
        st.update(lens=lens, nodes=nodes, pool=pool, table=table, cu=_cu(nodes),
                  starts=torch.tensor(lens, dtype=torch.int32, device="cuda"), parents=_parents(rng, nodes, case["chain"]),
                  q=_randn(g, sum(nodes), case["H"], d),
                  offset=_randn(g, case["H"], dtype=torch.float32) if case["sink"] == "learnable" else None)
        return st
    B, M, before = case["B"], case["most"], case["before"]
    lens = rng.integers(max(0, before - 60), before + 1, B)
    need = [(before + case["nodes"] + P - 1) // P] * B
    n_pages = sum(need) + 1
    st["pool"] = torch.randint(0, 256, (case["layers"], n_pages, H_kv, block), generator=g, device="cuda", dtype=torch.uint8)
    st["table"] = _table(g, need, n_pages)
    st["starts"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    kept = np.full((B, M), -1, dtype=np.int32)
    for b in range(B):
        n = int(rng.integers(0, M + 1))
        kept[b, :n] = np.sort(rng.permutation(case["nodes"])[:n])
    st["kept"] = torch.from_numpy(kept).cuda()
    return st


# ------------------------------------------------------------------------------------------ plain forms


def _rotate(x, c, s, case, back=False):
    """x [.., H, d] in 32 bits with its pairs turned by c, s [.., n] (the same rows, or the last of them shared)."""
    n, a = case["rot"] // 2, case["first"]
    c, s = c[..., None, :], s[..., None, :]
    if back:
        s = -s
    part = x[..., a:a + 2 * n]
    if case["interleaved"]:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2)
    else:
        x1, x2 = part[..., :n], part[..., n:]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    return torch.cat([x[..., :a], y, x[..., a + 2 * n:]], -1)


def _plain_rope(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]  # far positions: 64 bits
    table = torch.stack([angle.cos() * st["gain"], angle.sin() * st["gain"]], 1).float()
    c, s = table[:, 0], table[:, 1]
    out = [table] + [_rotate(st[n].float(), c, s, case).to(torch.bfloat16) for n in ("q", "k")]
    if case["train"]:
        out += [_rotate(st[n].float(), c, s, case, True).to(torch.bfloat16) for n in ("dq", "dk")]
    return out


def _quantise(x):
    """x [T, H, d] -> codes 0..15 [T, H, d] and scale bytes [T, H, d/16]."""
    T, H, d = x.shape
    f = x.float().view(T, H, d // 16, 16)
    r = f.abs().amax(-1)
    r = r / torch.full_like(r, 7.0)  # a quotient: a product with 1/7 would break ties
    u = r.contiguous().view(torch.int32)
    near = ((u + 0x7FFFF + ((u >> 20) & 1)) >> 20) - (112 << 3)  # to nearest, ties to even
    small = torch.round(r * 131072.0)  # below 2^-14 the format's step is 2^-17
    ok = torch.isfinite(f).all(-1)
    byte = torch.where(r < 2.0 ** -14, torch.nan_to_num(small).to(torch.int32), near).clamp(0, 0xF7)
    byte = torch.where(ok, byte, torch.full_like(byte, 0xFF))
    s = _scale_value(byte)[..., None]
    c = torch.where((s > 0) & ok[..., None], torch.round(f / s).clamp(-8, 7), torch.zeros_like(f)) + 8
    return c.to(torch.uint8).view(T, H, d), byte.to(torch.uint8)


def _scale_value(byte):
    return (byte.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _parts(pool, P):
    """The four parts of every page and head of a pool [n_pages, H_kv, block], as views."""
    n, H, block = pool.shape
    d = block * 8 // (9 * P)
    c, s = P * d // 2, P * d // 16
    return (pool[:, :, :c].view(n, H, P, d // 2), pool[:, :, c:2 * c].view(n, H, P // 2, 8, 2, d // 16),
            pool[:, :, 2 * c:2 * c + s].view(n, H, P, d // 16),
            pool[:, :, 2 * c + s:].view(n, H, P // 2, d // 16, 2), d)


def _slots(u, d):
    """Slots of the eighths 0..7 of the head dim for token pairs u: [n, 8]."""
    x = 2 * (u % 4) if d == 128 else 4 * ((u // 2) % 2)
    return torch.arange(8, device="cuda")[None, :] ^ x[:, None]


def _write(pool, pages, start, k, v, P):
    """Tokens start.. of one sequence into its pages."""
    T = k.shape[0]
    if T == 0:
        return
    pk, pv, sk, sv, d = _parts(pool, P)
    pos = torch.arange(start, start + T, device="cuda")
    pg, w = pages[pos // P].long(), pos % P
    ck, bk = _quantise(k)
    cv, bv = _quantise(v)
    H = k.shape[1]
    pk[pg, :, w] = ck[..., 0::2] | (ck[..., 1::2] << 4)
    sk[pg, :, w] = bk
    by = (cv[..., 0::2] | (cv[..., 1::2] << 4)).view(T, H, 8, d // 16)
    hh = torch.arange(H, device="cuda")
    pv[pg[:, None, None], hh[None, :, None], (w // 2)[:, None, None], _slots(w // 2, d)[:, None, :],
       (w % 2)[:, None, None]] = by
    sv[pg[:, None], hh[None, :], (w // 2)[:, None], :, (w % 2)[:, None]] = bv


def _read(pool, pages, start, T, P):
    """Tokens start.. of one sequence from its pages, in 32 bits: K, V [T, H, d]."""
    pk, pv, sk, sv, d = _parts(pool, P)
    pos = torch.arange(start, start + T, device="cuda")
    pg, w = pages[pos // P].long(), pos % P
    H = pool.shape[1]
    hh = torch.arange(H, device="cuda")

    def values(by, sc):
        c = torch.stack([by & 15, by >> 4], -1).view(T, H, d // 16, 16).float() - 8.0
        return (c * _scale_value(sc)[..., None]).view(T, H, d)

    kb = pk[pg, :, w]
    vb = pv[pg[:, None, None], hh[None, :, None], (w // 2)[:, None, None], _slots(w // 2, d)[:, None, :],
            (w % 2)[:, None, None]].reshape(T, H, d // 2)
    return (values(kb, sk[pg, :, w]), values(vb, sv[pg[:, None], hh[None, :], (w // 2)[:, None], :, (w % 2)[:, None]]))


def _plain_append(st):
    """Keys are rounded to bf16 after the rotation, as a rotation of its own would leave them."""
    case, P = st["case"], st["case"]["page"]
    c, s = st["rope"][:, 0], st["rope"][:, 1]
    q = _rotate(st["q"].float(), c, s, case).to(torch.bfloat16)
    k = _rotate(st["k"].float(), c, s, case).to(torch.bfloat16)
    ks, vs, at = [], [], 0
    for b, n in enumerate(st["lens"]):
        _write(st["pool"], st["table"][b], st["before"], k[at:at + n], st["v"][at:at + n], P)
        at += n
    for b, n in enumerate(st["lens"]):
        kk, vv = _read(st["pool"], st["table"][b], st["before"], n, P)
        ks.append(kk.to(torch.bfloat16))
        vs.append(vv.to(torch.bfloat16))
    return [q, torch.cat(ks), torch.cat(vs)]


def _ancestors(parents):
    """Steps from node i up to node a as [n, n], -1 where a is neither i nor an ancestor of it; depths [n]."""
    n = parents.shape[0]
    i = torch.arange(n, device="cuda")
    reach = ((parents[:, None] == i) | (i[:, None] == i)).float()  # itself and its parent
    for _ in range(max(1, n - 1).bit_length()):  # twice as far up each time
        reach = torch.matmul(reach, reach).clamp(max=1.0)
    depth = reach.sum(1).long() - 1
    return torch.where(reach > 0, depth[:, None] - depth, torch.full_like(depth, -1)), depth


def _seen(L, parents, window):
    """Truth values [n, L + n]: which tokens each node sees."""
    up, depth = _ancestors(parents)
    j = torch.arange(L, device="cuda")[None, :]
    before = (j >= L + depth[:, None] - window) if window >= 0 else torch.ones((len(depth), L), dtype=torch.bool, device="cuda")
    tree = (up >= 0) & ((up <= window) if window >= 0 else (up >= 0))
    return torch.cat([before, tree], 1)


def _plain_tree(st):
    case = st["case"]
    P, H, H_kv, d = case["page"], case["H"], case["H_kv"], case["d"]
    G, scale = H // H_kv, 1.0 / math.sqrt(d)
    T = sum(st["nodes"])
    o = torch.zeros((T, H, d), device="cuda")
    lse = torch.zeros((H, T), device="cuda")
    at = 0
    for b, (L, n) in enumerate(zip(st["lens"], st["nodes"])):
        rows = slice(at, at + n)
        k, v = _read(st["pool"], st["table"][b], 0, L + n, P)
        q = st["q"][rows].float().view(n, H_kv, G, d).permute(1, 2, 0, 3)  # [H_kv, G, n, d]
        s = torch.matmul(q.reshape(H_kv, G * n, d), k.permute(1, 2, 0)).view(H_kv, G, n, L + n) * scale
        s.masked_fill_(~_seen(L, st["parents"][rows], case["window"]), -math.inf)
        m = s.amax(-1)
        sink = None
        if case["sink"] != "vanilla":
            sink = (st["offset"] if case["sink"] == "learnable" else torch.zeros(H, device="cuda")).view(H_kv, G, 1)
            m = torch.maximum(m, sink)
        e = torch.exp(s - m[..., None])
        del s
        l = e.sum(-1)
        if sink is not None:
            l = l + torch.exp(sink - m)
        ob = torch.matmul(e.view(H_kv, G * n, L + n), v.transpose(0, 1)).view(H_kv, G, n, d) / l[..., None]
        o[rows] = ob.permute(2, 0, 1, 3).reshape(n, H, d)
        lse[:, rows] = (m + torch.log(l)).view(H, n)
        at += n
    return [o.to(torch.bfloat16), lse]


def _places(st):
    """Page and place in it of every move's source and destination."""
    P = st["case"]["page"]
    b, i = torch.nonzero(st["kept"] >= 0, as_tuple=True)
    src, dst = st["starts"].long()[b] + st["kept"].long()[b, i], st["starts"].long()[b] + i
    return st["table"].long()[b, src // P], src % P, st["table"].long()[b, dst // P], dst % P


def _plain_keep(st):
    """Nodes are kept in ascending order, so no source is a destination of an earlier move."""
    P = st["case"]["page"]
    n_layers, n_pages, H, block = st["pool"].shape
    pg, w, pg2, w2 = _places(st)
    layer = torch.arange(n_layers, device="cuda")[:, None] * n_pages
    pg, pg2 = (layer + pg).flatten(), (layer + pg2).flatten()
    w, w2 = w.repeat(n_layers), w2.repeat(n_layers)
    pk, pv, sk, sv, d = _parts(st["pool"].view(-1, H, block), P)
    hh = torch.arange(H, device="cuda")[None, :]

    def at_v(pg, w):
        return (pg[:, None, None], hh[..., None], (w // 2)[:, None, None], _slots(w // 2, d)[:, None, :], (w % 2)[:, None, None])

    k, ks, v = pk[pg, :, w], sk[pg, :, w], pv[at_v(pg, w)]
    vs = sv[pg[:, None], hh, (w // 2)[:, None], :, (w % 2)[:, None]]
    pk[pg2, :, w2], sk[pg2, :, w2], pv[at_v(pg2, w2)] = k, ks, v
    sv[pg2[:, None], hh, (w2 // 2)[:, None], :, (w2 % 2)[:, None]] = vs
    return [st["pool"]]


# ------------------------------------------------------------------------------------------ the framework's calls


def _own(st):
    import scaled_dot_product_tmem_gb300 as sdpa
    case, op = st["case"], st["case"]["op"]
    if op in ("rope", "append"):
        kw = dict(interleaved=case["interleaved"], first_dim=case["first"])
    if op == "rope":
        table = sdpa.rope_table(st["inv_freq"], st["positions"], gain=st["gain"])
        out = [table, *sdpa.rope_forward(st["q"], st["k"], table, **kw)]
        if case["train"]:
            out += sdpa.rope_backward(st["dq"], st["dk"], table, **kw)
        return out
    if op == "append":
        q = sdpa.kv4_append_rope(st["q"], st["k"], st["v"], st["rope"], st["cu"], st["pool"], st["table"], st["starts"], **kw)
        return [q, *sdpa.kv4_gather(st["pool"], st["table"], st["cu"], st["starts"], st["k"].shape[0], case["d"])]
    if op == "tree":
        return list(sdpa.sdpa_tree_kv4(st["q"], st["cu"], st["parents"], st["pool"], st["table"], st["starts"],
                                       window=case["window"], softmax_type=case["sink"], softmax_offset=st["offset"]))
    sdpa.attn_kv4_keep(st["pool"], st["table"], st["starts"], st["kept"], case["d"])
    return [st["pool"]]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree, "keep": _plain_keep}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ 64 bits


def _exact_turned(x, angle, gain, case, sign=1.0):
    """Pairs of x [.., H, d] as complex numbers times gain exp(sign i angle), angle [.., n]."""
    n, a = case["rot"] // 2, case["first"]
    f = torch.arange(n, device="cuda")
    i1, i2 = (a + 2 * f, a + 2 * f + 1) if case["interleaved"] else (a + f, a + n + f)
    x = x.double()
    z = torch.complex(x[..., i1], x[..., i2]) * torch.polar(torch.full_like(angle, gain), sign * angle)[..., None, :]
    y = x.clone()
    y[..., i1], y[..., i2] = z.real, z.imag
    return y


def _exact_rope(case, seed):
    st = prepare(case, seed)
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    out = [torch.stack([angle.cos(), angle.sin()], 1) * st["gain"]]
    out += [_exact_turned(st[n], angle, st["gain"], case) for n in ("q", "k")]
    if case["train"]:
        out += [_exact_turned(st[n], angle, st["gain"], case, -1.0) for n in ("dq", "dk")]
    return out


def _pow2(e):
    """2^e in 64 bits for whole e, from the number's bits (a power function may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_held(x):
    """What 16 values are held as, in 64 bits."""
    f = x.double().view(*x.shape[:-1], -1, 16)
    r = f.abs().amax(-1)
    r = r / torch.full_like(r, 7)  # a quotient here too
    e = torch.clamp(torch.frexp(r)[1] - 1, -14, 15)  # exponent of the format's binade
    step = _pow2(e - 3)
    s = torch.clamp(torch.round(r / step) * step, max=61440.0)[..., None]
    c = torch.clamp(torch.round(f / torch.where(s > 0, s, torch.ones_like(s))), -8, 7)
    return torch.where(s > 0, c * s, torch.zeros_like(f)).view(x.shape)


def _exact_append(case, seed):
    st = prepare(case, seed)
    w, _ = _frequencies(case["rot"])
    start = int(case["before"])
    pos = torch.cat([torch.arange(n, device="cuda") for n in st["lens"]]) + start
    angle = pos.double()[:, None] * w
    q, k = (_exact_turned(st[n], angle, 1.0, case) for n in ("q", "k"))
    return [q, _exact_held(k.to(torch.bfloat16)), _exact_held(st["v"])]


def _exact_cache(pool, pages, T, P, d):
    """K and V of T tokens from their pages in 64 bits, by byte addresses."""
    dev, H = pool.device, pool.shape[1]
    p = torch.arange(T, device=dev).view(T, 1, 1)
    flat = pool.view(-1)
    base = (pages[p // P].long() * H + torch.arange(H, device=dev).view(1, H, 1)) * pool.shape[2]
    x = torch.arange(d, device=dev).view(1, 1, d)
    w = p % P
    u, g = w // 2, x // (d // 8)
    slot = g ^ (2 * (u % 4) if d == 128 else 4 * ((u // 2) % 2))
    at_k = w * (d // 2) + x // 2
    at_v = P * d // 2 + u * d + slot * (d // 8) + (w % 2) * (d // 16) + (x % (d // 8)) // 2
    at_sk = P * d + w * (d // 16) + x // 16
    at_sv = P * d + P * d // 16 + u * (d // 8) + (x // 16) * 2 + w % 2
    out = []
    for at, sc in ((at_k, at_sk), (at_v, at_sv)):
        c = (flat[base + at].long() >> (4 * (x % 2))) & 15
        sb = flat[base + sc].long()
        e, m = sb >> 3, (sb & 7).double()
        s = torch.where(e > 0, (1 + m / 8) * _pow2(e - 15), (m / 8) * _pow2(e - 14))
        out.append((c - 8).double() * s)
    return out


def _exact_tree(case, seed):
    st = prepare(case, seed)
    if work(case)["flops"] > 2e12:
        return None
    H, G, d, P, w = case["H"], case["H"] // case["H_kv"], case["d"], case["page"], case["window"]
    T = sum(st["nodes"])
    o = torch.zeros((T, H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, T), dtype=torch.float64, device="cuda")
    parents, at = st["parents"].tolist(), 0
    for b, (L, n) in enumerate(zip(st["lens"], st["nodes"])):
        seen = np.zeros((n, L + n), dtype=bool)
        for i in range(n):
            path, a = [], i
            while a >= 0:
                path.append(a)
                a = parents[at + a]
            depth = len(path) - 1
            seen[i, L + np.array(path if w < 0 else path[:w + 1])] = True
            seen[i, max(0, L + depth - w) if w >= 0 else 0:L] = True
        seen = torch.from_numpy(seen).cuda()
        pages = st["table"][b]
        for hk in range(case["H_kv"]):
            few = st["pool"][pages[:(L + n + P - 1) // P].long(), hk:hk + 1].contiguous()
            k, v = (t[:, 0] for t in _exact_cache(few, torch.arange(few.shape[0], device="cuda"), L + n, P, d))
            for h in range(hk * G, (hk + 1) * G):
                s = (st["q"][at:at + n, h].double() @ k.T) / math.sqrt(d)
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
                if case["sink"] != "vanilla":
                    z = st["offset"][h].double() if case["sink"] == "learnable" else s.new_zeros(())
                    s = torch.cat([s, z.expand(n, 1)], 1)
                z = torch.logsumexp(s, 1)
                o[at:at + n, h], lse[h, at:at + n] = torch.exp(s[:, :L + n] - z[:, None]) @ v, z
        at += n
    return [o, lse]


def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    st = prepare(case, seed)
    new = st["pool"].clone()  # byte by byte, in order, from the addresses
    P, d = case["page"], case["d"]
    b, i = (t.tolist() for t in torch.nonzero(st["kept"] >= 0, as_tuple=True))
    kept, starts, table = st["kept"].tolist(), st["starts"].tolist(), st["table"].tolist()

    def bytes_of(w):
        u, g, x = w // 2, np.arange(8)[:, None], np.arange(d // 16)
        slot = g ^ (2 * (u % 4) if d == 128 else 4 * ((u // 2) % 2))
        return torch.from_numpy(np.concatenate([
            w * (d // 2) + np.arange(d // 2), (P * d // 2 + u * d + slot * (d // 8) + (w % 2) * (d // 16) + x).ravel(),
            P * d + w * (d // 16) + x, P * d + P * d // 16 + u * (d // 8) + 2 * x + w % 2])).cuda()

    places = [bytes_of(w) for w in range(P)]
    for s, r in zip(b, i):
        src, dst = starts[s] + kept[s][r], starts[s] + r
        new[:, table[s][dst // P], :, places[dst % P]] = new[:, table[s][src // P], :, places[src % P]]
    return [new]
