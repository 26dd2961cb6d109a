"""The dense-path operators of the library, as cases to time and compare.

Four operators, in the order a serving loop calls them: the per-head norm and
rotation of a batch's queries and keys, the attention of a chunk of new tokens
over the paged cache, the attention weight each micro-block of the cache
received, and the eviction of the blocks that received least.

``own`` chooses between their plain form (elementary torch operations in 32
bits) and the library's calls.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
HEADS = ((32, 4), (8, 2), (16, 16), (12, 4))  # (query heads, KV heads)
PLAIN_SCORES = 1 << 29  # scores that the plain forms hold at once


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token of one sequence, fused projection output: latency alone
        dict(name="norm-rope 1 token", op="norm", N=1, Hq=32, Hk=4, D=128, rot=128, pairs=False,
             fused=True),
        # the indexer's query heads and key of a decode batch, adjacent pairs, half the dims rotated
        dict(name="norm-rope indexer b128", op="norm", N=128, Hq=16, Hk=1, D=64, rot=32, pairs=True,
             fused=False),
        # a prompt chunk, an odd number of tokens
        dict(name="norm-rope 16k", op="norm", N=16381, Hq=32, Hk=4, D=128, rot=128, pairs=False,
             fused=True),
        # one token of two short contiguous-size sequences (the tiny preset's heads and lengths)
        dict(name="attend 1 token tiny", op="attend", S=2, L=4099, Lmin=1500, T=1, Hq=8, Hkv=2,
             P=64, ragged=True),
        # a dense decode step of the b32x32k preset
        dict(name="attend 1 token b32x32k", op="attend", S=32, L=32768, Lmin=32768, T=1, Hq=32,
             Hkv=4, P=64, ragged=False),
        # ragged chunks behind ragged contexts, a page size that does not divide a tile
        dict(name="attend ragged chunks", op="attend", S=9, L=9001, Lmin=517, T=700, Hq=32, Hkv=4,
             P=48, ragged=True),
        # a prompt chunk of 4,096 tokens that ends a 65,536-token context
        dict(name="attend 4k chunk at 64k", op="attend", S=1, L=65536, Lmin=65536, T=4096, Hq=32,
             Hkv=4, P=64, ragged=False),
        # the weights of one decode token over the b32x32k preset
        dict(name="mass 1 token b32x32k", op="mass", S=32, L=32768, Lmin=32768, T=1, Hq=32, Hkv=4,
             P=64, ragged=False),
        # the weights that the newest rows of ragged prompts gave
        dict(name="mass ragged chunks", op="mass", S=5, L=30011, Lmin=1027, T=300, Hq=32, Hkv=4,
             P=64, ragged=True),
        # every row of an 8,192-token prompt
        dict(name="mass 8k prompt", op="mass", S=1, L=8192, Lmin=8192, T=8192, Hq=32, Hkv=4, P=64,
             ragged=False),
        # one short sequence down to 1,024 tokens
        dict(name="evict 4k to 1k", op="evict", S=1, L=4099, Lmin=4099, keep=256, sink=1, recent=16,
             Hkv=2, di=64, P=64, ragged=False),
        # a ragged batch down to 8,192 tokens a sequence
        dict(name="evict b24 to 8k", op="evict", S=24, L=65536, Lmin=1024, keep=2048, sink=1,
             recent=64, Hkv=4, di=128, P=64, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "attend", "attend", "mass", "evict"))
    if op == "norm":
        D = rng.choice((64, 128))
        Hq, Hk = rng.choice(((32, 4), (8, 2), (16, 1), (16, 16), (12, 4)))
        return dict(op=op, N=_log_int(rng, 1, 16000), Hq=Hq, Hk=Hk, D=D,
                    rot=rng.choice((16, 32, 64, D)), pairs=rng.random() < 0.5,
                    fused=rng.random() < 0.5)
    Hq, Hkv = rng.choice(HEADS)
    P = rng.choice((4, 16, 20, 32, 48, 64, 128, 256))
    ragged = rng.random() < 0.7
    if op == "evict":
        L = _log_int(rng, 300, 65536)
        S = _log_int(rng, 1, min(24, max(1, 1500000 // L)))
        keep = max(8, _log_int(rng, 32, max(40, L // 5)))
        return dict(op=op, S=S, L=L, Lmin=max(1, L // 7) if ragged else L, keep=keep,
                    sink=rng.randint(0, 3), recent=rng.randint(1, max(1, keep // 3)),
                    Hkv=rng.choice((2, 4, 8)), di=rng.choice((64, 128)), P=P, ragged=ragged)
    L = _log_int(rng, 64, 65536)
    S = _log_int(rng, 1, min(64, max(1, 1000000 // L)))
    # rows x heads x tokens stay below the largest listed case of the operator
    most = (4000 * 32 * 65536 if op == "attend" else 8192 * 32 * 4000) // (S * Hq * L)
    T = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, min(most, L, 4096, 60000 // S)))
    return dict(op=op, S=S, L=L, Lmin=max(T, L // 9) if ragged else L, T=T, Hq=Hq, Hkv=Hkv, P=P,
                ragged=ragged)


def lengths(case):
    """(context lengths, chunk lengths) of a case's sequences; the first sequence has the largest of both."""
    S, L, lo, T = case["S"], case["L"], case["Lmin"], case.get("T", 0)
    r = random.Random(S * 1000003 + L)
    lens, chunks = [L], [T]
    for _ in range(S - 1):
        lens.append(int(round(math.exp(r.uniform(math.log(lo), math.log(L))))) if case["ragged"] else L)
        chunks.append(min(lens[-1], r.randint(1, T)) if case["ragged"] and T > 1 else T)
    return lens, chunks


# ------------------------------------------------------------------ inputs

def _randn(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    out.normal_(0.0, scale, generator=g)
    return out


def _table(lens, P, seed, first=0):
    """Shuffled pages for the sequences, from page `first` on: (block table, end of the page ids)."""
    pages = [-(-n // P) for n in lens]
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    ids = torch.randperm(sum(pages), generator=g).to(torch.int32) + first
    width = max(pages)
    rows = [torch.nn.functional.pad(x, (0, width - x.numel()), value=-1) for x in ids.split(pages)]
    return torch.stack(rows).to(DEV), first + sum(pages)


def _heads(case):
    from types import SimpleNamespace
    return SimpleNamespace(Hq=case.get("Hq", case["Hkv"]), Hkv=case["Hkv"], D=128,
                           Hi=4, di=case.get("di", 64), P=case["P"], scale=1.0 / math.sqrt(128.0))


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "norm":
        N, Hq, Hk, D, rot = (case[x] for x in ("N", "Hq", "Hk", "D", "rot"))
        if case["fused"]:  # views of a projection that holds q, k and v of a token side by side
            qkv = _randn((N, Hq + 2 * Hk, D), seed, 2.0)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            st["q"], st["k"] = _randn((N, Hq, D), seed, 2.0), _randn((N, Hk, D), seed + 71, 2.0)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 5)
        st["qw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        st["kw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        max_pos = 65536
        st["pos"] = torch.randint(0, max_pos, (N,), generator=g, device=DEV, dtype=torch.int32)
        freq = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
        ang = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * freq
        st["rope"] = torch.cat((ang.cos(), ang.sin()), 1).float()
        if own:  # outputs that a serving loop keeps
            st["out"] = (torch.empty((N, Hq, D), dtype=torch.bfloat16, device=DEV),
                         torch.empty((N, Hk, D), dtype=torch.bfloat16, device=DEV))
        return st
    lens, chunks = lengths(case)
    d = st["dims"] = _heads(case)
    st["table"], used = _table(lens, d.P, seed)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["op"] == "evict":
        nb = [-(-n // 4) for n in lens]
        kept = [min(4 * case["keep"], n) for n in lens]
        st["dst"], pages = _table(kept, d.P, seed + 1, used)
        width = st["table"].shape[1]
        st["dst"] = torch.nn.functional.pad(st["dst"], (0, width - st["dst"].shape[1]), value=-1)
        st["first"] = used
        st["k"] = _randn((pages, d.P, d.Hkv, 128), seed)
        st["v"] = _randn((pages, d.P, d.Hkv, 128), seed + 1)
        st["x"] = _randn((pages, d.P, d.di), seed + 2)
        st["side"] = _randn((pages, d.P // 4, d.di), seed + 3)
        for t in ("k", "v", "x", "side"):
            st[t][used:] = 0
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 4)
        # weights as attention gives them: over many octaves, and equal ones
        m = torch.randn((case["S"], max(nb)), generator=g, device=DEV).mul_(2.0).exp_()
        st["mass"] = torch.where(m < 0.1, torch.full_like(m, 0.0625), m)
    else:
        st["start"] = torch.tensor([sum(chunks[:i]) for i in range(len(chunks) + 1)],
                                   dtype=torch.int32, device=DEV)
        st["k"] = _randn((used, d.P, d.Hkv, 128), seed)
        st["q"] = _randn((sum(chunks), d.Hq, 128), seed + 2, 2.0)
        if case["op"] == "attend":
            st["v"] = _randn((used, d.P, d.Hkv, 128), seed + 1)
        else:
            st["v"] = st["k"]
            st["lse"] = _attend(st, weights=False)[1]
            g = torch.Generator(device=DEV)
            g.manual_seed(seed + 4)
            st["mass"] = torch.rand((case["S"], -(-max(lens) // 4)), generator=g, device=DEV)
        st["x"] = torch.zeros((used, d.P, d.di), dtype=torch.bfloat16, device=DEV)
        st["side"] = torch.zeros((used, d.P // 4, d.di), dtype=torch.bfloat16, device=DEV)
    if own:  # the cache's handle, and the outputs and scratch that a serving loop keeps
        from block_sparse_decode_b200 import qsa
        st["qd"] = qsa.QsaDims.of(d)
        st["cache"] = qsa.QsaCache(st["k"], st["v"], st["x"], st["side"], st["table"])
        if case["op"] == "attend":
            st["buf"] = qsa.alloc_chunk_attention(st["qd"], case["S"], sum(chunks), device=DEV)
        elif case["op"] == "mass":
            st["buf"] = qsa.alloc_attention_mass(st["qd"], case["S"], sum(chunks),
                                                 st["mass"].shape[1], device=DEV)
        else:
            st["buf"] = qsa.alloc_evict(case["S"], st["mass"].shape[1], case["keep"], device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _norm_rope(x, w, eps, cos, sin, pairs):
    """[N, H, D] -> normed and rotated; cos, sin [N, 1, rot / 2]."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w
    r = cos.shape[-1]
    if pairs:
        a, b = y[..., 0:2 * r:2], y[..., 1:2 * r:2]
    else:
        a, b = y[..., :r], y[..., r:2 * r]
    c, d = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((c, d), -1).flatten(-2) if pairs else torch.cat((c, d), -1)
    return torch.cat((head, y[..., 2 * r:]), -1).to(x.dtype)


def _parts(S, heads, G, T, L):
    """Sequence ranges and KV-head ranges whose scores fit in the plain forms' memory."""
    n = max(1, PLAIN_SCORES // max(1, heads * G * T * L))
    h = heads if n > 1 else max(1, min(heads, PLAIN_SCORES // max(1, G * T * L)))
    return [(s, min(S, s + n), k, min(heads, k + h)) for s in range(0, S, n)
            for k in range(0, heads, h)]


def _scores(st, s0, s1, h0, h1):
    """Scaled scores [n, h, G, T, L] of a range, -inf where a row does not see a token, with
    the rows' place in the chunk order [n, T], which are rows, and the tokens' pool rows."""
    d, case = st["dims"], st["case"]
    T, G, P = case["T"], d.Hq // d.Hkv, d.P
    lens, start = st["lens"].long(), st["start"].long()
    L = case["L"]
    tok = torch.arange(L, device=DEV)
    page = st["table"][s0:s1].long()[:, tok // P].clamp_min(0)
    at = page * P + tok % P                                   # [n, L]
    k = st["k"].flatten(0, 1)[:, h0:h1][at].float()           # [n, L, h, D]
    i = torch.arange(T, device=DEV)
    count = (start[s0 + 1:s1 + 1] - start[s0:s1])[:, None]    # [n, 1]
    is_row = i[None] < count
    row = torch.where(is_row, start[s0:s1, None] + i, 0)
    q = st["q"][row].view(s1 - s0, T, d.Hkv, G, 128)[:, :, h0:h1].float()
    z = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3), k.permute(0, 2, 3, 1))
    z = z.view(s1 - s0, h1 - h0, G, T, L).mul_(d.scale)
    see = lens[s0:s1, None] - count + i + 1                   # tokens that a row sees
    z.masked_fill_(tok >= torch.where(is_row, see, 0)[:, None, None, :, None], -math.inf)
    return z, row, is_row, at


def _attend(st, weights=True):
    d, T = st["dims"], st["case"]["T"]
    G = d.Hq // d.Hkv
    Nq = st["q"].shape[0]
    out = torch.zeros((Nq, d.Hkv, G, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((Nq, d.Hkv, G), device=DEV)
    for s0, s1, h0, h1 in _parts(st["case"]["S"], d.Hkv, G, T, st["case"]["L"]):
        z, row, is_row, at = _scores(st, s0, s1, h0, h1)
        m = z.amax(-1, keepdim=True).clamp_min(-1e30)
        p = z.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        rows = row[is_row]
        lse[rows, h0:h1] = (m + total.log())[..., 0].permute(0, 3, 1, 2)[is_row]
        if weights:
            v = st["v"].flatten(0, 1)[:, h0:h1][at].float().permute(0, 2, 1, 3)  # [n, h, L, D]
            o = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:4], 128) / total
            out[rows, h0:h1] = o.permute(0, 3, 1, 2, 4)[is_row].to(out.dtype)
    return out.view(Nq, d.Hq, 128), lse.view(Nq, d.Hq)


def _mass(st):
    d, case = st["dims"], st["case"]
    G, T, L = d.Hq // d.Hkv, case["T"], case["L"]
    lse = st["lse"].view(-1, d.Hkv, G)
    mass = st["mass"].clone()
    nb = -(-L // 4)
    for s0, s1, h0, h1 in _parts(case["S"], d.Hkv, G, T, L):
        z, row, _, _ = _scores(st, s0, s1, h0, h1)
        p = z.sub_(lse[row][:, :, h0:h1].permute(0, 2, 3, 1)[..., None]).exp_()
        w = torch.nn.functional.pad(p.sum((1, 2, 3)), (0, 4 * nb - L))
        mass[s0:s1] += w.view(s1 - s0, nb, 4).sum(-1)
    return mass


def _evict(st):
    case, d, P = st["case"], st["dims"], st["dims"].P
    keep, mass, lens = case["keep"], st["mass"], st["lens"].long()
    nb = (lens + 3) // 4
    j = torch.arange(mass.shape[1], device=DEV)
    always = (j < case["sink"]) | (j >= nb[:, None] - case["recent"])
    key = torch.where(always, math.inf, mass)
    key = torch.where(j < nb[:, None], key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    n = nb.clamp_max(keep)
    i = torch.arange(order.shape[1], device=DEV)
    order = torch.where(i < n[:, None], order, mass.shape[1]).sort(1).values
    kept = torch.where(i < n[:, None], order, -1)
    src = kept.clamp_min(0)
    kept_mass = torch.where(i < n[:, None], mass.gather(1, src), 0.0)
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[1]), value=-1).int()
    new_mass = torch.nn.functional.pad(kept_mass, (0, mass.shape[1] - kept_mass.shape[1]))
    new_lens = 4 * n - (4 * nb - lens)
    # token rows of the pools, from the old place to the new one
    t = torch.arange(4 * i.numel(), device=DEV)
    live = t < new_lens[:, None]
    old = 4 * src.repeat_interleave(4, 1) + t % 4

    def rows(table, pos, per):
        seq = torch.arange(table.shape[0], device=DEV)[:, None]
        page = table.long()[seq, torch.where(pos < table.shape[1] * per, pos // per, 0)]
        return page * per + pos % per

    a = rows(st["table"], old, P)[live]
    b = rows(st["dst"], t.expand_as(old), P)[live]
    for pool in (st["k"], st["v"], st["x"]):
        flat = pool.flatten(0, 1)
        flat[b] = flat[a]
    full = i < (new_lens // 4)[:, None]  # a partial block has no key in the side pool
    side = st["side"].flatten(0, 1)
    side[rows(st["dst"], i.expand_as(src), P // 4)[full]] = side[rows(st["table"], src, P // 4)[full]]
    return kept, new_lens.int(), new_mass


def _evicted(st, kept, new_lens, new_mass):
    n = st["first"]
    return {"kept": kept, "lens": new_lens, "mass": new_mass, "k": st["k"][n:], "v": st["v"][n:],
            "x": st["x"][n:], "side": st["side"][n:]}


def run(st):
    case = st["case"]
    if case["op"] == "norm":
        if own:
            from block_sparse_decode_b200 import qsa
            q, k = st["out"]
            qsa.qsa_qk_norm_rope(st["pos"], st["q"], st["k"], st["qw"], st["kw"], 1e-6,
                                 st["rope"], q, k, interleaved=case["pairs"])
            return q, k
        t = st["rope"][st["pos"].long()][:, None]
        cos, sin = t.chunk(2, -1)
        return (_norm_rope(st["q"], st["qw"], 1e-6, cos, sin, case["pairs"]),
                _norm_rope(st["k"], st["kw"], 1e-6, cos, sin, case["pairs"]))
    if case["op"] == "attend":
        if own:
            from block_sparse_decode_b200 import qsa
            b = st["buf"]
            qsa.qsa_chunk_attention(st["qd"], st["cache"], st["lens"], st["start"], st["q"],
                                    b.out, b.lse, b.ws)
            return b.out, b.lse
        return _attend(st)
    if case["op"] == "mass":
        if own:
            from block_sparse_decode_b200 import qsa
            b = st["buf"]
            qsa.qsa_attention_mass(st["qd"], st["cache"], st["lens"], st["start"], st["q"],
                                   st["lse"], st["mass"], b.mass, b.ws)
            return b.mass
        return _mass(st)
    if own:
        from block_sparse_decode_b200 import qsa
        b = st["buf"]
        qsa.qsa_evict(st["qd"], st["cache"], st["lens"], st["mass"], case["keep"], case["sink"],
                      case["recent"], st["dst"], b.kept, b.new_lens, b.mass, b.ws)
        return _evicted(st, b.kept, b.new_lens, b.mass)
    return _evicted(st, *_evict(st))


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "norm":
        values = case["N"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 4 * values + case["N"] * (4 + 4 * case["rot"]) + 8 * case["D"],
                "flops": 8 * values}
    lens, chunks = lengths(case)
    if case["op"] == "evict":
        kept = [min(4 * case["keep"] - (-n) % 4, n) for n in lens]
        token = 2 * case["Hkv"] * 256 + 2 * case["di"]
        blocks = [-(-n // 4) for n in lens]
        moved = sum(n * token + n // 4 * 2 * case["di"] for n in kept)
        return {"bytes": 2 * moved + 4 * sum(blocks) + 4 * case["S"] * (case["keep"] + max(blocks)),
                "flops": sum(blocks)}
    pairs = sum(T * (n - T) + T * (T + 1) // 2 for n, T in zip(lens, chunks)) * case["Hq"]
    cached = sum(lens) * case["Hkv"] * 256
    rows = sum(chunks) * case["Hq"]
    if case["op"] == "attend":
        return {"bytes": 2 * cached + rows * (512 + 4), "flops": 512 * pairs}
    return {"bytes": cached + rows * (256 + 4) + 2 * sum(-(-n // 4) for n in lens) * 4,
            "flops": 256 * pairs}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        rot = case["rot"]
        res = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            x = x.double()
            n = (x.pow(2).sum(-1) / case["D"] + 1e-6).sqrt()
            y = x / n[..., None] * w.double()
            z = y.clone()
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + rot // 2)
                ang = (st["pos"].double() * 1e6 ** (-2.0 * i / rot))[:, None]
                z[..., a] = y[..., a] * ang.cos() - y[..., b] * ang.sin()
                z[..., b] = y[..., b] * ang.cos() + y[..., a] * ang.sin()
            res.append(z)
        return res
    lens, chunks = lengths(case)
    d = st["dims"]
    table = st["table"].cpu().long()
    if case["op"] == "evict":
        keep, width = case["keep"], st["mass"].shape[1]
        kept = torch.full((case["S"], keep), -1, dtype=torch.int32)
        mass = torch.zeros((case["S"], width), dtype=torch.float64)
        dst = st["dst"].cpu().long()
        pools = {t: torch.zeros_like(st[t][st["first"]:]).double() for t in ("k", "v", "x", "side")}
        new = []
        for s, n in enumerate(lens):
            m = st["mass"][s].cpu().tolist()
            nb = -(-n // 4)
            forced = set(range(min(nb, case["sink"]))) | set(range(max(0, nb - case["recent"]), nb))
            rest = sorted((b for b in range(nb) if b not in forced), key=lambda b: (-m[b], b))
            # where everything is forced in, the first ones stay
            mine = sorted((sorted(forced) + rest)[:keep])
            new.append(4 * len(mine) - (4 * nb - n))
            kept[s, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            mass[s, :len(mine)] = torch.tensor([m[b] for b in mine], dtype=torch.float64)
            to = torch.arange(new[-1])
            frm = 4 * torch.tensor(mine)[to // 4] + to % 4
            a, b = table[s, frm // d.P], dst[s, to // d.P] - st["first"]
            for t in ("k", "v", "x"):
                pools[t][b.to(DEV), (to % d.P).to(DEV)] = st[t][a.to(DEV), (frm % d.P).to(DEV)].double()
            to = torch.arange(new[-1] // 4)
            frm, R = torch.tensor(mine)[to], d.P // 4
            pools["side"][(dst[s, to // R] - st["first"]).to(DEV), (to % R).to(DEV)] = \
                st["side"][table[s, frm // R].to(DEV), (frm % R).to(DEV)].double()
        return {"kept": kept.to(DEV), "lens": torch.tensor(new, dtype=torch.int32, device=DEV),
                "mass": mass.to(DEV), **pools}
    G, row = d.Hq // d.Hkv, 0
    out = torch.zeros((sum(chunks), d.Hq, 128), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(chunks), d.Hq), dtype=torch.float64, device=DEV)
    if case["op"] == "mass":
        mass = st["mass"].double()
    for s, (n, T) in enumerate(zip(lens, chunks)):
        pages = st["table"][s, :-(-n // d.P)].long()
        K, V = (st[t][pages].flatten(0, 1)[:n].double() for t in ("k", "v"))
        for r0 in range(0, T, 256):
            r1 = min(T, r0 + 256)
            sees = torch.arange(n, device=DEV) <= torch.arange(n - T + r0, n - T + r1, device=DEV)[:, None]
            for h in range(d.Hq):
                z = st["q"][row + r0:row + r1, h].double() @ K[:, h // G].T * d.scale
                if case["op"] == "mass":
                    w = torch.exp(z - st["lse"][row + r0:row + r1, h, None].double()) * sees
                    w = torch.nn.functional.pad(w.sum(0), (0, (-n) % 4))
                    mass[s, :w.numel() // 4] += w.view(-1, 4).sum(1)
                else:
                    e = torch.logsumexp(z.masked_fill(~sees, -math.inf), 1)
                    lse[row + r0:row + r1, h] = e
                    out[row + r0:row + r1, h] = (torch.exp(z - e[:, None]) * sees) @ V[:, h // G]
        row += T
    return mass if case["op"] == "mass" else (out, lse)
