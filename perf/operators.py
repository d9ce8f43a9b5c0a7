"""Cases of the packed-sequence attention and of the 4-bit paged key/value cache.

Five operators of a serving and training stack around fused attention:

  fwd     attention over packed sequences of different lengths (no padding rows)
  train   the same, forward and backward
  append  new keys and values quantised to 4 bits into the pages of a cache, and read back
  decode  attention of a sequence's newest tokens over its 4-bit cache
  copy    pages of a cache copied (forks, copy-on-write) or moved (compaction)

`run` computes each either with elementary torch operations in 32 bits (`own` false) or through
this package's entry points (`own` true).  `exact` gives the same outputs from the definitions
in 64 bits.

The cache.  A pool holds pages [n_pages, H_kv, block]; the block of one page and one head holds
P tokens of head dim d as four consecutive parts:
  K codes   [P][d/2]            two codes a byte, the even dim in the low nibble
  V codes   [P/2][8][2][d/16]   token pair u, eighth g of the head dim at slot g ^ x(u), the two tokens
  K scales  [P][d/16]           one byte for 16 dims
  V scales  [P/2][d/16][2]
with x(u) = 2 (u mod 4) at d = 128 and 4 (floor(u / 2) mod 2) at d = 64.  A code c in 0..15 stands
for (c - 8) s; a scale byte holds bits 14..7 of a half-precision number (5 exponent bits, 3
mantissa bits, no sign).  For 16 values x, s = max|x| / 7 rounded to that format (ties to even,
at most 0xF7) and c = 8 + clamp(round(x / s), -8, 7); 16 values with an infinity or NaN among
them get s = 0xFF (NaN).
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # a handful of short requests of a small model: what counts is the launch
        dict(name="fwd_short_d64", op="fwd", lens="1,37,128,5", lens_kv="", H=8, H_kv=2, d_qk=64, d_v=64, causal=True,
             window=-1, sink="vanilla"),
        # a prefill batch under a sliding window with a learnable sink
        dict(name="fwd_swa_sink", op="fwd", lens="2048,1333,700,64,2048,511,1000,257", lens_kv="", H=32, H_kv=8,
             d_qk=128, d_v=128, causal=True, window=1024, sink="learnable"),
        # a batch of prompts, one of them long
        dict(name="fwd_prompts", op="fwd", lens="16384,8192,4099,2047,1024,700,64,1", lens_kv="", H=32, H_kv=8,
             d_qk=128, d_v=128, causal=True, window=-1, sink="vanilla"),
        # training on short packed documents
        dict(name="train_docs_d64", op="train", lens="200,77,512,130,333,1,64,259", lens_kv="", H=16, H_kv=16,
             d_qk=64, d_v=64, causal=True, window=-1, sink="off_by_one"),
        # training on long packed documents
        dict(name="train_packed", op="train", lens="8192,3001,2048,1500,900,650,93", lens_kv="", H=32, H_kv=8, d_qk=128,
             d_v=128, causal=True, window=-1, sink="vanilla"),
        # one token for each of many running requests enters the cache
        dict(name="append_step", op="append", lens=",".join(["1"] * 64), before="37", H_kv=8, d=128, page=16),
        # prompts enter the cache
        dict(name="append_prompts", op="append", lens="8192,4097,2000,1024,333,31", before="5", H_kv=8, d=128, page=64),
        # one running request of a small model
        dict(name="decode_single_d64", op="decode", lens="200", S_q=1, H=8, H_kv=2, d=64, page=16, window=-1,
             sink="vanilla"),
        # a batch of running requests of different age
        dict(name="decode_batch", op="decode",
             lens="4096,1,777,8191,2500,64,65,3999,1200,5000,31,6144,900,2047,16,7000", S_q=1, H=32, H_kv=8, d=128,
             page=64, window=-1, sink="vanilla"),
        # long contexts, two tokens at a time (a proposed token is checked with the last one)
        dict(name="decode_long", op="decode", lens="131072,65536,100001,32768", S_q=2, H=32, H_kv=8, d=128, page=64,
             window=-1, sink="vanilla"),
        # a few requests fork: the last, partly filled page of each is copied
        dict(name="copy_fork", op="copy", pages=12, n_pages=512, layers=1, H_kv=8, d=128, page=16),
        # the pool of several layers is compacted
        dict(name="copy_compact", op="copy", pages=1500, n_pages=4096, layers=4, H_kv=8, d=128, page=64),
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
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["fwd", "train", "append", "decode", "copy"])
    if op in ("fwd", "train"):
        H, H_kv = rng.choice([(32, 8), (8, 2), (16, 16), (32, 1), (12, 4), (7, 7)])
        d_qk, d_v = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        causal = rng.random() < 0.8
        lens = _draw_lens(rng, 24, 8000 if op == "fwd" else 5000, 16000 if op == "fwd" else 9000)
        kv = ""
        if rng.random() < 0.3:  # queries and keys of different lengths, some entries without keys
            kv = ",".join(str(max(0, int(v) + rng.randint(-int(v), int(v)))) for v in lens.split(","))
        case = dict(op=op, lens=lens, lens_kv=kv, H=H, H_kv=H_kv, d_qk=d_qk, d_v=d_v, causal=causal,
                    window=_log_int(rng, 1, 2048) if causal and rng.random() < 0.4 else -1,
                    sink=rng.choice(["vanilla", "off_by_one", "learnable"]))
        return case
    H, H_kv = rng.choice([(32, 8), (8, 2), (16, 16), (32, 1), (24, 4), (64, 8), (7, 7)])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        return dict(op=op, lens=_draw_lens(rng, 64, 8000, 15000), before=str(rng.randint(0, 300)), H_kv=H_kv, d=d,
                    page=page)
    if op == "decode":
        return dict(op=op, lens=_draw_lens(rng, 64, 60000, 250000), S_q=rng.choice([1, 1, 1, 2, 3, 5]), H=H, H_kv=H_kv,
                    d=d, page=page, window=_log_int(rng, 1, 4096) if rng.random() < 0.3 else -1,
                    sink=rng.choice(["vanilla", "off_by_one", "learnable"]))
    n_pages = _log_int(rng, 64, 4000)
    return dict(op="copy", pages=_log_int(rng, 1, n_pages // 3), n_pages=n_pages, layers=rng.randint(1, 4), H_kv=H_kv,
                d=d, page=page)


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def _pairs(lq, lk, causal, window):
    """Visible (query, key) pairs of one sequence, key j seen by query i when j <= i and j >= i - window."""
    if not causal:
        return lq * lk
    i = np.arange(lq, dtype=np.int64)
    hi = np.minimum(i, lk - 1)
    lo = np.maximum(0, i - window) if window >= 0 else np.zeros_like(i)
    return int(np.maximum(0, hi - lo + 1).sum())


def work(case):
    op = case["op"]
    if op in ("fwd", "train"):
        lq, lk = _ints(case["lens"]), _ints(case["lens_kv"]) or _ints(case["lens"])
        H, H_kv, dq, dv = case["H"], case["H_kv"], case["d_qk"], case["d_v"]
        pairs = sum(_pairs(a, b, case["causal"], case["window"]) for a, b in zip(lq, lk))
        q, k, v, o = 2 * sum(lq) * H * dq, 2 * sum(lk) * H_kv * dq, 2 * sum(lk) * H_kv * dv, 2 * sum(lq) * H * dv
        flops = 2 * pairs * H * (dq + dv)
        byts = q + k + v + o + 4 * sum(lq) * H
        if op == "train":  # dO read, dQ dK dV written; S, dP, dV, dK, dQ products
            byts += o + q + k + v
            flops += 2 * pairs * H * (3 * dq + 2 * dv)
        return dict(bytes=byts, flops=flops)
    token = case["d"] * 9 // 8  # bytes of one token and head: codes and scales of K and V
    if op == "append":  # read, packed, read back
        n = sum(_ints(case["lens"])) * case["H_kv"]
        return dict(bytes=n * (2 * 4 * case["d"] + 2 * token), flops=n * 2 * case["d"] * 4)
    if op == "decode":
        lens, w, s = _ints(case["lens"]), case["window"], case["S_q"]
        seen = [min(l, w + s) if w >= 0 else l for l in lens]
        rows = len(lens) * s * case["H"]
        return dict(bytes=sum(seen) * case["H_kv"] * token + rows * (4 * case["d"] + 4),
                    flops=4 * sum(seen) * s * case["H"] * case["d"])
    return dict(bytes=2 * case["pages"] * case["layers"] * case["H_kv"] * case["page"] * token, flops=0)


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


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case=case)
    if op in ("fwd", "train"):
        lq = _ints(case["lens"])
        lk = _ints(case["lens_kv"]) or lq
        st.update(lq=lq, lk=lk, q=_randn(g, sum(lq), case["H"], case["d_qk"]),
                  k=_randn(g, sum(lk), case["H_kv"], case["d_qk"]), v=_randn(g, sum(lk), case["H_kv"], case["d_v"]),
                  cu_q=_cu(lq), cu_kv=_cu(lk))
        st["offset"] = _randn(g, case["H"], dtype=torch.float32) if case["sink"] == "learnable" else None
        if op == "train":
            st["dout"] = _randn(g, sum(lq), case["H"], case["d_v"])
        return st
    H_kv, d, P = case["H_kv"], case["d"], case["page"]
    block = P * d * 9 // 8
    if op == "append":
        lens, before = _ints(case["lens"]), int(case["before"])
        need = [(before + n + P - 1) // P for n in lens]
        n_pages = sum(need) + 3
        st.update(lens=lens, before=before, k=_kv_like(g, sum(lens), H_kv, d, True),
                  v=_kv_like(g, sum(lens), H_kv, d, False), cu=_cu(lens), table=_table(g, need, n_pages),
                  starts=torch.full((len(lens),), before, dtype=torch.int32, device="cuda"),
                  pool=torch.randint(0, 256, (n_pages, H_kv, block), generator=g, device="cuda", dtype=torch.uint8))
        return st
    if op == "decode":
        lens = _ints(case["lens"])
        need = [(n + P - 1) // P for n in lens]
        n_pages = sum(need) + 1
        pool = torch.randint(0, 256, (n_pages, H_kv, block), generator=g, device="cuda", dtype=torch.uint8)
        table = _table(g, need, n_pages)
        for b, n in enumerate(lens):
            k, v = _kv_like(g, n, H_kv, d, True), _kv_like(g, n, H_kv, d, False)
            _write(pool, table[b], 0, k, v, P)
        st.update(lens=lens, pool=pool, table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  q=_randn(g, len(lens), case["S_q"], case["H"], d),
                  offset=_randn(g, case["H"], dtype=torch.float32) if case["sink"] == "learnable" else None)
        return st
    n_pages = case["n_pages"]
    st["pool"] = torch.randint(0, 256, (case["layers"], n_pages, H_kv, block), generator=g, device="cuda",
                               dtype=torch.uint8)
    perm = np.random.default_rng(seed).permutation(n_pages)[:2 * case["pages"]].astype(np.int32)
    st["src"], st["dst"] = torch.from_numpy(perm[:case["pages"]].copy()), torch.from_numpy(perm[case["pages"]:].copy())
    return st


# ------------------------------------------------------------------------------------------ plain forms


def _masked(Lq, Lk, causal, window, r0, r1):
    """Truth values [r1 - r0, Lk]: which keys rows r0..r1-1 do not see."""
    i = torch.arange(r0, r1, device="cuda")[:, None]
    j = torch.arange(Lk, device="cuda")[None, :]
    out = torch.zeros((r1 - r0, Lk), dtype=torch.bool, device="cuda")
    if causal:
        out = j > i
        if window >= 0:
            out = out | (j < i - window)
    return out


def _sink(case, st, heads):
    """The sink's logit of each head in `heads` as [n, 1], or None."""
    if case["sink"] == "vanilla":
        return None
    if case["sink"] == "off_by_one":
        return torch.zeros((len(heads), 1), device="cuda")
    return st["offset"][heads][:, None]


def _softmax(s, sink):
    """Row-wise probabilities and log of the denominator, over s [h, r, n] and the sink's logit."""
    m = s.amax(-1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf, device=s.device, dtype=s.dtype)
    if sink is not None:
        m = torch.maximum(m, sink)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m0[..., None])
    l = e.sum(-1)
    if sink is not None:
        l = l + torch.exp(sink - m0)
    p = torch.where(l[..., None] > 0, e / l[..., None], torch.zeros_like(e))
    return p, m0 + torch.log(l)


def _row_step(H, Lk):
    """Query rows at a time, so that a block of scores stays near 4 GB."""
    return max(1, (1 << 30) // max(1, H * Lk))


def _plain_packed(st):
    """One sequence, one kv head's group of query heads and one block of rows at a time."""
    case = st["case"]
    H, H_kv, dq, dv = case["H"], case["H_kv"], case["d_qk"], case["d_v"]
    G, scale = H // H_kv, 1.0 / math.sqrt(dq)
    train = case["op"] == "train"
    Tq, Tk = st["q"].shape[0], st["k"].shape[0]
    o = torch.zeros((Tq, H, dv), device="cuda")
    lse = torch.zeros((H, Tq), device="cuda")
    if train:
        gq, gk, gv = (torch.zeros(t.shape, device="cuda") for t in (st["q"], st["k"], st["v"]))
        goff = torch.zeros(H, device="cuda")
    aq = ak = 0
    for Lq, Lk in zip(st["lq"], st["lk"]):
        for hk in range(H_kv):
            hs = list(range(hk * G, (hk + 1) * G))
            k, v = st["k"][ak:ak + Lk, hk].float(), st["v"][ak:ak + Lk, hk].float()
            sink = _sink(case, st, hs)
            step = _row_step(G, Lk)
            for r0 in range(0, Lq, step):
                r1 = min(Lq, r0 + step)
                q = st["q"][aq + r0:aq + r1, hs].float().transpose(0, 1)
                s = torch.matmul(q, k.t()) * scale
                s.masked_fill_(_masked(Lq, Lk, case["causal"], case["window"], r0, r1), -math.inf)
                p, z = _softmax(s, sink)
                del s
                ob = torch.matmul(p, v)
                o[aq + r0:aq + r1, hs] = ob.transpose(0, 1)
                lse[hs, aq + r0:aq + r1] = z
                if train:
                    do = st["dout"][aq + r0:aq + r1, hs].float().transpose(0, 1)
                    D = (do * ob).sum(-1)
                    gv[ak:ak + Lk, hk] += torch.matmul(p.transpose(1, 2), do).sum(0)
                    ds = p * (torch.matmul(do, v.t()) - D[..., None])
                    gq[aq + r0:aq + r1, hs] = (torch.matmul(ds, k) * scale).transpose(0, 1)
                    gk[ak:ak + Lk, hk] += torch.matmul(ds.transpose(1, 2), q).sum(0) * scale
                    if case["sink"] == "learnable":
                        ps = torch.where(torch.isinf(z), torch.zeros_like(z), torch.exp(sink - z))
                        goff[hs] -= (ps * D).sum(-1)
        aq, ak = aq + Lq, ak + Lk
    out = [o.to(torch.bfloat16), lse]
    if train:
        out += [t.to(torch.bfloat16) for t in (gq, gk, gv)]
        if case["sink"] == "learnable":
            out.append(goff)
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
    case, P = st["case"], st["case"]["page"]
    ks, vs, at = [], [], 0
    for b, n in enumerate(st["lens"]):
        _write(st["pool"], st["table"][b], st["before"], st["k"][at:at + n], st["v"][at:at + n], P)
        at += n
    for b, n in enumerate(st["lens"]):
        k, v = _read(st["pool"], st["table"][b], st["before"], n, P)
        ks.append(k.to(torch.bfloat16))
        vs.append(v.to(torch.bfloat16))
    return [torch.cat(ks), torch.cat(vs)]


def _plain_decode(st):
    case = st["case"]
    P, H, H_kv, d, S = case["page"], case["H"], case["H_kv"], case["d"], case["S_q"]
    G, scale = H // H_kv, 1.0 / math.sqrt(d)
    B = len(st["lens"])
    o = torch.zeros((B, S, H, d), device="cuda")
    lse = torch.zeros((B, H, S), device="cuda")
    for b, L in enumerate(st["lens"]):
        k, v = _read(st["pool"], st["table"][b], 0, L, P)
        q = st["q"][b].float().view(S, H_kv, G, d).permute(1, 2, 0, 3).reshape(H_kv, G * S, d)
        s = torch.matmul(q, k.permute(1, 2, 0)) * scale  # [H_kv, G S, L], row g S + s
        i = L - S + torch.arange(S, device="cuda").repeat(G)[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        bad = j > i
        if case["window"] >= 0:
            bad = bad | (j < i - case["window"])
        s.masked_fill_(bad, -math.inf)
        sink = _sink(case, st, list(range(H)))
        if sink is not None:
            sink = sink.view(H_kv, G, 1).expand(H_kv, G, S).reshape(H_kv, G * S)
        p, z = _softmax(s, sink)
        ob = torch.matmul(p, v.transpose(0, 1)).view(H_kv, G, S, d)
        o[b] = ob.permute(2, 0, 1, 3).reshape(S, H, d)
        lse[b] = z.view(H, S)
    return [o.to(torch.bfloat16), lse]


def _plain_copy(st):
    src, dst = st["src"].cuda().long(), st["dst"].cuda().long()
    st["pool"][:, dst] = st["pool"][:, src]
    return [st["pool"]]


# ------------------------------------------------------------------------------------------ the framework's calls


def _own(st):
    import scaled_dot_product_tmem_gb300 as sdpa
    case, op = st["case"], st["case"]["op"]
    if op in ("fwd", "train"):
        kw = dict(causal=case["causal"], window=case["window"], softmax_type=case["sink"],
                  softmax_offset=st["offset"])
        o, lse = sdpa.sdpa_forward_packed(st["q"], st["k"], st["v"], st["cu_q"], st["cu_kv"], **kw)
        out = [o, lse]
        if op == "train":
            dq, dk, dv, d_off = sdpa.sdpa_backward_packed(st["q"], st["k"], st["v"], o, st["dout"], lse, st["cu_q"],
                                                          st["cu_kv"], **kw)
            out += [dq, dk, dv]
            if case["sink"] == "learnable":
                out.append(d_off)
        return out
    if op == "append":
        sdpa.attn_kv4_append(st["k"], st["v"], st["cu"], st["pool"], st["table"], st["starts"])
        return list(sdpa.kv4_gather(st["pool"], st["table"], st["cu"], st["starts"], st["k"].shape[0], case["d"]))
    if op == "decode":
        return list(sdpa.sdpa_decode_kv4(st["q"], st["pool"], st["table"], st["seq_lens"], window=case["window"],
                                         softmax_type=case["sink"], softmax_offset=st["offset"]))
    sdpa.attn_kv4_copy_pages(st["pool"], st["src"], st["dst"])
    return [st["pool"]]


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_packed, "train": _plain_packed, "append": _plain_append, "decode": _plain_decode,
            "copy": _plain_copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ 64 bits


def _exact_rows(q, k, v, sink, scale, seen):
    """One head in 64 bits: seen(i, j) truth values; returns o, log-denominator, probabilities."""
    s = (q @ k.T) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    if sink is not None:
        s = torch.cat([s, sink.double().expand(s.shape[0], 1)], 1)
    if s.shape[1] == 0:
        return q.new_zeros(q.shape[0], v.shape[1]), q.new_full((q.shape[0],), -math.inf), s
    z = torch.logsumexp(s, 1)
    p = torch.where(torch.isinf(z)[:, None], torch.zeros_like(s), torch.exp(s - z[:, None]))[:, :k.shape[0]]
    return p @ v, z, p


def _exact_packed(case, seed):
    st = prepare(case, seed)
    w = work(case)
    if w["flops"] * 2 > 12e12:  # 64-bit products of the largest cases take too long
        return None
    train = case["op"] == "train"
    H, G, scale = case["H"], case["H"] // case["H_kv"], case["d_qk"] ** -0.5
    q, k, v = (st[n].double() for n in "qkv")
    o = q.new_zeros(q.shape[0], H, case["d_v"])
    lse = q.new_zeros(H, q.shape[0])
    dq, dk, dv, doff = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), q.new_zeros(H)
    ends_q, ends_k = np.cumsum([0] + st["lq"]), np.cumsum([0] + st["lk"])
    for b in range(len(st["lq"])):
        rk = slice(int(ends_k[b]), int(ends_k[b + 1]))
        for h in range(H):
            sink = {"vanilla": None, "off_by_one": q.new_zeros(1)}.get(case["sink"], None)
            if case["sink"] == "learnable":
                sink = st["offset"][h:h + 1].double()
            kk, vv = k[rk, h // G], v[rk, h // G]
            for a in range(0, st["lq"][b], 4096):
                z = min(a + 4096, st["lq"][b])
                rq = slice(int(ends_q[b]) + a, int(ends_q[b]) + z)
                # under a causal mask no row of the block sees a key at or past z
                n = min(kk.shape[0], z) if case["causal"] else kk.shape[0]
                i = torch.arange(a, z, device="cuda").view(-1, 1)
                j = torch.arange(n, device="cuda").view(1, -1)
                seen = torch.ones((z - a, n), dtype=torch.bool, device="cuda")
                if case["causal"]:
                    seen = (j <= i) & ((i - j <= case["window"]) if case["window"] >= 0 else seen)
                ob, lb, p = _exact_rows(q[rq, h], kk[:n], vv[:n], sink, scale, seen)
                o[rq, h], lse[h, rq] = ob, lb
                if train:
                    g = st["dout"][rq, h].double()
                    dv[rk, h // G][:n] += p[:, :n].T @ g
                    ds = p[:, :n] * (g @ vv[:n].T - (g * ob).sum(1, keepdim=True))
                    dq[rq, h] = ds @ kk[:n] * scale
                    dk[rk, h // G][:n] += ds.T @ q[rq, h] * scale
                    if case["sink"] == "learnable":
                        doff[h] -= (torch.exp(sink - lb) * (g * ob).sum(1)).sum()
    out = [o, lse]
    if train:
        out += [dq, dk, dv]
        if case["sink"] == "learnable":
            out.append(doff)
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


def _exact_decode(case, seed):
    st = prepare(case, seed)
    S, H, G, d = case["S_q"], case["H"], case["H"] // case["H_kv"], case["d"]
    o = torch.zeros((len(st["lens"]), S, H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((len(st["lens"]), H, S), dtype=torch.float64, device="cuda")
    for b, L in enumerate(st["lens"]):
        for hk in range(case["H_kv"]):
            k, v = _exact_head(st, b, hk, L)
            i = torch.arange(L - S, L, device="cuda").view(-1, 1)
            j = torch.arange(L, device="cuda").view(1, -1)
            seen = (j <= i) & ((i - j <= case["window"]) if case["window"] >= 0 else (j >= 0))
            for h in range(hk * G, (hk + 1) * G):
                sink = {"vanilla": None, "off_by_one": o.new_zeros(1)}.get(case["sink"], None)
                if case["sink"] == "learnable":
                    sink = st["offset"][h:h + 1].double()
                o[b, :, h], lse[b, h], _ = _exact_rows(st["q"][b, :, h].double(), k, v, sink, d ** -0.5, seen)
    return [o, lse]


def _exact_head(st, b, hk, L):
    """K and V [L, d] of one sequence and kv head in 64 bits."""
    case = st["case"]
    pages = st["table"][b]
    n = (L + case["page"] - 1) // case["page"]
    few = st["pool"][pages[:n].long(), hk:hk + 1]
    k, v = _exact_cache(few.contiguous(), torch.arange(max(n, 1), device="cuda"), L, case["page"], case["d"])
    return k[:, 0], v[:, 0]


def exact(case, seed):
    op = case["op"]
    if op in ("fwd", "train"):
        return _exact_packed(case, seed)
    if op == "append":
        st = prepare(case, seed)
        return [_exact_held(st["k"]), _exact_held(st["v"])]
    if op == "decode":
        return _exact_decode(case, seed)
    st = prepare(case, seed)
    new = st["pool"].clone()
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        new[:, b] = st["pool"][:, a]
    return [new]
