"""The dense path and the eviction on the GPU (through the C ABI) against their
formulas in 64 bits: norm + rotation, chunk attention over the paged cache,
attention weight per micro-block, eviction, and the four in a loop with the
append and the decode step.

Tolerances count roundings: a bf16 store or operand is off by at most 2^-8 of
its value (half a step), fp32 sums by far less. An attention output then is
off by the rounding of its weights to bf16, 2^-8 of sum_t w_t |V_t|, and its
own, 2^-8 of itself; 2^-12 of the first covers the fp32 part (scores of at
most 128 products, the exponential, the sums).
"""

from __future__ import annotations

import math

import pytest
import torch

from block_sparse_decode_b200 import qsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = 2.0 ** -8  # half a bf16 step


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


# ------------------------------------------------------------ norm + rotation

def norm_rope_ref(x, w, eps, pos, freq, pairs):
    """[N, H, D] in 64 bits; also the size of each rotated pair (for tolerances)."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    z, size = y.clone(), y.abs()
    rot = 2 * len(freq)
    if rot:
        a = torch.arange(rot // 2, device=DEV)
        ia, ib = (2 * a, 2 * a + 1) if pairs else (a, a + rot // 2)
        ang = pos.double()[:, None, None] * freq
        z[..., ia] = y[..., ia] * ang.cos() - y[..., ib] * ang.sin()
        z[..., ib] = y[..., ib] * ang.cos() + y[..., ia] * ang.sin()
        size[..., ia] = size[..., ib] = torch.hypot(y[..., ia], y[..., ib])
    return z, size


@pytest.mark.parametrize("N,Hq,Hk,D,rot,pairs,fused", [
    (1, 32, 4, 128, 128, False, True), (3, 8, 2, 128, 64, True, False),
    (257, 12, 4, 128, 16, False, True), (33, 16, 1, 64, 64, True, True),
    (1025, 5, 3, 64, 32, False, False), (700, 32, 4, 128, 128, True, True),
    (5, 1, 0, 64, 16, False, False), (40, 7, 9, 128, 0, False, True),
    (2000, 32, 4, 128, 128, False, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(N, Hq, Hk, D, rot, pairs, fused, norm):
    if fused:
        qkv = randn((N, Hq + 2 * Hk + 1, D), N, 3.0)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk] if Hk else None
    else:
        q, k = randn((N, Hq, D), N, 3.0), randn((N, Hk, D), N + 1) if Hk else None
    max_pos = 300000
    g = torch.Generator(device=DEV)
    g.manual_seed(N)
    pos = torch.randint(0, max_pos, (N,), generator=g, device=DEV, dtype=torch.int32)
    pos[0] = max_pos - 1
    if N > 2:
        pos[1] = -1  # padding
    freq = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / max(rot, 1))
    rope = qsa.rope_table(max_pos, rot, 1e6) if rot else None
    qw = torch.rand(D, generator=g, device=DEV) + 0.5 if norm else None
    kw = torch.rand(D, generator=g, device=DEV) - 0.5 if norm else None
    q_out = torch.full((N, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((N, Hk, D), 7.0, dtype=torch.bfloat16, device=DEV) if Hk else None
    qsa.qsa_qk_norm_rope(pos, q, k, qw, kw, 1e-6, rope, q_out, k_out, interleaved=pairs)
    assert qsa.qsa_check_device_errors() == 0
    live = pos >= 0
    for x, w, out in ((q, qw, q_out), (k, kw, k_out)):
        if x is None:
            continue
        ref, size = norm_rope_ref(x, w, 1e-6, pos, freq, pairs)
        # one rounding; 2^-20 of the pair covers the fp32 norm and rotation
        tol = HALF * ref.abs() + 2.0 ** -20 * size + 1e-30
        assert bool(((out.double() - ref).abs() <= tol)[live].all())
        assert bool((out[~live] == 7.0).all())
        if x.is_contiguous():  # in place gives the same bits
            y = x.clone()
            qsa.qsa_qk_norm_rope(pos, y, None, w, None, 1e-6, rope, y, interleaved=pairs)
            assert torch.equal(y[live], out[live]) and torch.equal(y[~live], x[~live])


def test_norm_rope_position_out_of_range():
    q = randn((4, 2, 64), 1)
    out = torch.zeros_like(q)
    pos = torch.tensor([0, 8, 7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    qsa.qsa_qk_norm_rope(pos, q, None, None, None, 0.0, qsa.rope_table(8, 64), out)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert e.value.status == qsa.QSA_ERR_BOUNDS and "flags=64" in str(e.value)
    assert bool((out[[1, 3]] == 0).all()) and torch.equal(out[0], q[0])
    assert qsa.qsa_check_device_errors() == 0


# ------------------------------------------------------------ a paged cache

class Paged:
    """Sequences of random K, V and indexer keys in shuffled pages; every slot
    that no token holds is NaN. `spare` pages behind them belong to nobody."""

    def __init__(self, lens, Hq=32, Hkv=4, P=64, di=64, seed=0, spare=0, scale=1.0, width=None):
        self.dims = qsa.QsaDims(Hq, Hkv, 128, 4, di, P, 1 / math.sqrt(128.0))
        self.lens = lens
        pages = [-(-n // P) for n in lens]
        total = sum(pages) + 3
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed))[:sum(pages)]
        width = width or max(max(pages), 1)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for s, ids in enumerate(perm.split(pages)):
            table[s, :len(ids)] = ids
        self.cache = qsa.alloc_cache(self.dims, total + spare, table, DEV)
        self.first_spare = total
        c = self.cache
        for t in (c.k_pool, c.v_pool, c.kidx_pool, c.side_pool):
            t.fill_(math.nan)
        self.k, self.v, self.x, self.side = [], [], [], []
        for s, n in enumerate(lens):
            self.k.append(randn((n, Hkv, 128), seed + 10 * s + 1, scale))
            self.v.append(randn((n, Hkv, 128), seed + 10 * s + 2))
            self.x.append(randn((n, di), seed + 10 * s + 3))
            self.side.append(randn((n // 4, di), seed + 10 * s + 4))
            page, slot = self.places(table.to(DEV), s, n, P)
            c.k_pool[page, slot], c.v_pool[page, slot] = self.k[s], self.v[s]
            c.kidx_pool[page, slot] = self.x[s]
            page, slot = self.places(table.to(DEV), s, n // 4, P // 4)
            c.side_pool[page, slot] = self.side[s]
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    @staticmethod
    def places(table, s, n, per):
        t = torch.arange(n, device=DEV)
        return table[s].long()[t // per], t % per

    def rows(self, chunks, seed, scale=1.0, extra=0):
        start = [0]
        for T in chunks:
            start.append(start[-1] + T)
        q = randn((start[-1] + extra, self.dims.Hq, 128), seed, scale)
        return torch.tensor(start, dtype=torch.int32, device=DEV), q


def attention_ref(pc, chunks, q):
    """out, lse, sum of w |V|, and the weight of every token, in 64 bits."""
    d, G, row = pc.dims, pc.dims.Hq // pc.dims.Hkv, 0
    out = torch.zeros((sum(chunks), d.Hq, 128), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(chunks), d.Hq), dtype=torch.float64, device=DEV)
    size, mass = torch.zeros_like(out), []
    for s, (n, T) in enumerate(zip(pc.lens, chunks)):
        w_tok = torch.zeros(n, dtype=torch.float64, device=DEV)
        for h in range(d.Hq):
            z = q[row:row + T, h].double() @ pc.k[s][:, h // G].double().T * d.scale
            see = torch.arange(n, device=DEV) <= torch.arange(n - T, n, device=DEV)[:, None]
            z = z.masked_fill(~see, -math.inf)
            e = torch.logsumexp(z, 1)
            w = torch.exp(z - e[:, None])
            lse[row:row + T, h] = e
            out[row:row + T, h] = w @ pc.v[s][:, h // G].double()
            size[row:row + T, h] = w @ pc.v[s][:, h // G].double().abs()
            w_tok += w.sum(0)
        mass.append(torch.nn.functional.pad(w_tok, (0, (-n) % 4)).view(-1, 4).sum(1))
        row += T
    return out, lse, size, mass


CHUNKS = [
    # (context lengths, chunk lengths, Hq, Hkv, P)
    ([1], [1], 32, 4, 64),
    ([5], [5], 8, 2, 64),
    ([4099, 1500], [1, 1], 8, 2, 64),
    ([130, 129, 128, 127, 1], [1, 1, 1, 1, 1], 32, 4, 64),
    ([300, 77, 640], [300, 0, 33], 32, 4, 64),
    ([1000, 33, 257], [17, 16, 257], 32, 4, 48),
    ([515, 70], [40, 9], 12, 4, 20),
    ([515, 70], [90, 70], 16, 16, 16),
    ([700], [129], 21, 3, 4),
    ([700, 13], [64, 13], 10, 2, 128),
    ([2050, 9], [65, 1], 6, 1, 256),
    ([5000, 4000], [31, 200], 32, 4, 1024),
    ([20011, 3, 9000], [2, 3, 1], 32, 4, 64),
]


@pytest.mark.parametrize("lens,chunks,Hq,Hkv,P", CHUNKS)
def test_chunk_attention_and_mass(lens, chunks, Hq, Hkv, P):
    pc = Paged(lens, Hq, Hkv, P, seed=len(lens) + lens[0], scale=2.0)
    start, q = pc.rows(chunks, 5, 1.5)
    S, Nq = len(lens), sum(chunks)
    b = qsa.alloc_chunk_attention(pc.dims, S, Nq, out_dtype=torch.float32)
    b.ws.random_(0, 255)  # the scratch needs no initialisation
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    ref, lse, size, mass = attention_ref(pc, chunks, q)
    assert bool(((b.out.double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6).all())
    assert float((b.lse.double() - lse).abs().max()) <= 1e-3
    out16 = torch.empty((Nq, Hq, 128), dtype=torch.bfloat16, device=DEV)
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, out16, None, b.ws)
    assert torch.equal(out16, b.out.to(torch.bfloat16))  # the same, rounded once

    ld = qsa.ld_for(lens) + 3
    base = torch.rand((S, ld), device=DEV)
    m = qsa.alloc_attention_mass(pc.dims, S, Nq, ld)
    m.ws.random_(0, 255)
    lse32 = lse.float().contiguous()
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse32, base, m.mass, m.ws)
    assert qsa.qsa_check_device_errors() == 0
    for s, want in enumerate(mass):
        got = m.mass[s].double()
        full = torch.nn.functional.pad(want, (0, ld - want.numel()))
        # scores of up to 128 fp32 products of size ~10: 1e-3 of a weight
        assert bool(((got - base[s].double() - full).abs() <= 1e-3 * full + 1e-6).all())
        assert torch.equal(m.mass[s, want.numel():], base[s, want.numel():])
    # in place and again: the same bits; no mass_in: from zero
    again = base.clone()
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse32, again, again, m.ws)
    assert torch.equal(again, m.mass)
    zero = torch.full_like(base, math.nan)
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse32, None, zero, m.ws)
    assert bool(((zero + base - m.mass).abs() <= 1e-5 * m.mass.abs()).all())


def test_chunk_attention_leaves_other_rows():
    """Rows behind the last chunk, and a chunk longer than its sequence, stay as
    they were; the others are computed."""
    pc = Paged([100, 40, 300], seed=3)
    start, q = pc.rows([10, 41, 20], 5, extra=6)
    out = torch.full((77, 32, 128), 5.0, device=DEV)
    lse = torch.full((77, 32), 5.0, device=DEV)
    ws = qsa.alloc_chunk_attention(pc.dims, 3, 77).ws
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, out, lse, ws)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert "flags=16" in str(e.value)
    assert bool((out[10:51] == 5).all()) and bool((lse[10:51] == 5).all())
    assert bool((out[71:] == 5).all()) and bool((lse[71:] == 5).all())
    one = Paged([100, 300], seed=3)
    one.k, one.v = [pc.k[0], pc.k[2]], [pc.v[0], pc.v[2]]
    rows = torch.cat((torch.arange(10), torch.arange(51, 71))).to(DEV)
    ref, ref_lse, size, _ = attention_ref(one, [10, 20], q[rows])
    assert bool(((out[rows].double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6).all())
    assert float((lse[rows].double() - ref_lse).abs().max()) <= 1e-3
    mass = torch.full((3, 80), 2.0, device=DEV)
    mws = qsa.alloc_attention_mass(pc.dims, 3, 77, 80).ws
    lse[10:51] = -math.inf
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse, mass, mass, mws)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert "flags=16" in str(e.value)
    assert bool((mass[1] == 2).all()) and abs(float((mass[0] - 2).sum()) - 320) < 0.5


def test_bad_page_is_flagged():
    pc = Paged([200, 90], seed=4)
    pc.cache.block_table[0, 1] = pc.cache.k_pool.shape[0]
    start, q = pc.rows([2, 3], 6)
    b = qsa.alloc_chunk_attention(pc.dims, 2, 5)
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert "flags=2" in str(e.value)
    ref, lse, size, _ = attention_ref(pc, [2, 3], q)
    assert float((b.lse[2:].double() - lse[2:]).abs().max()) <= 1e-3
    m = qsa.alloc_attention_mass(pc.dims, 2, 5, 50)
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse.float(), None, m.mass,
                           m.ws)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert "flags=2" in str(e.value)


def test_large_scores_and_ties():
    """Scores of size 1,000 that grow along the context (the running maximum
    moves in every tile), and equal scores."""
    pc = Paged([1025, 700], 8, 2, 64, seed=8)
    start, q = pc.rows([3, 40], 9)
    q[:] = 1.0
    for s, n in enumerate(pc.lens):
        pc.k[s] = (torch.linspace(-9, 9, n, device=DEV)[:, None, None] *
                   torch.ones((n, 2, 128), device=DEV)).to(torch.bfloat16)
        if s == 1:
            pc.k[s] = torch.zeros_like(pc.k[s])
        page, slot = pc.places(pc.cache.block_table, s, n, 64)
        pc.cache.k_pool[page, slot] = pc.k[s]
    q = (q * 8).contiguous()
    b = qsa.alloc_chunk_attention(pc.dims, 2, 43, out_dtype=torch.float32)
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    ref, lse, size, _ = attention_ref(pc, [3, 40], q)
    # these scores are sums of equal products, whose fp32 sums are off by
    # at most 128 * 2^-24 of 9 * 8 * 128 * scale = 815: 6e-3 of a score and,
    # where two tokens share the weight, of the weights
    assert bool(((b.out.double() - ref).abs() <= (HALF + 2 ** -6) * size + 1e-6).all())
    assert float((b.lse.double() - lse).abs().max()) <= 1e-2


# ------------------------------------------------------------ eviction

def evict_ref(lens, mass, keep, sink, recent):
    kept = []
    for s, n in enumerate(lens):
        nb = -(-n // 4)
        m = [(-math.inf if math.isnan(v) else v) for v in mass[s].tolist()[:nb]]
        forced = [j for j in range(nb) if j < sink or j >= nb - recent]
        rest = sorted((j for j in range(nb) if sink <= j < nb - recent), key=lambda j: (-m[j], j))
        kept.append(list(range(nb)) if nb <= keep else sorted(forced + rest[:keep - len(forced)]))
    return kept


@pytest.mark.parametrize("lens,keep,sink,recent,P,Hkv,di,kind", [
    ([4099], 256, 1, 16, 64, 2, 64, "wide"),
    ([0, 1, 2, 3, 4, 5, 31, 33], 8, 1, 2, 16, 1, 64, "wide"),
    ([1000, 1001, 1002, 1003, 40], 100, 3, 7, 48, 4, 128, "ties"),
    ([9001, 20000], 1700, 0, 1, 20, 3, 64, "all equal"),
    ([515, 333], 20, 4, 16, 4, 2, 128, "wide"),  # every kept block is forced
    ([70000, 640], 5000, 1, 64, 128, 4, 64, "nan"),
    ([257, 511], 500, 0, 1, 64, 2, 64, "wide"),  # nothing to evict
    ([8200], 1, 0, 1, 1024, 2, 64, "wide"),
])
def test_evict(lens, keep, sink, recent, P, Hkv, di, kind):
    S = len(lens)
    pc = Paged(lens, 4 * Hkv, Hkv, P, di, seed=keep, spare=S * (-(-4 * keep // P)))
    ld = qsa.ld_for(lens) + 2
    g = torch.Generator(device=DEV)
    g.manual_seed(keep)
    mass = torch.randn((S, ld), generator=g, device=DEV).mul_(4).exp_()
    if kind == "ties":
        mass = torch.randint(0, 3, (S, ld), generator=g, device=DEV).float() - 1.0
        mass[mass == 0] = -0.0
        mass[:, ::2] += 0.0
    elif kind == "all equal":
        mass.fill_(0.25)
    elif kind == "nan":
        mass[:, ::3] = math.nan
        mass[:, 1::7] = math.inf
        mass[:, 2::9] = -math.inf
    width = pc.cache.block_table.shape[1]
    per = -(-4 * keep // P)
    dst = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(S * per, generator=torch.Generator().manual_seed(1)).view(S, per)
    dst[:, :min(per, width)] = ids[:, :width].to(DEV) + pc.first_spare
    b = qsa.alloc_evict(S, ld, keep)
    before = [t[:pc.first_spare].view(torch.int16).clone() for t in
              (pc.cache.k_pool, pc.cache.v_pool, pc.cache.kidx_pool, pc.cache.side_pool)]
    qsa.qsa_evict(pc.dims, pc.cache, pc.seq_lens, mass, keep, sink, recent, dst, b.kept,
                  b.new_lens, b.mass, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    c = pc.cache
    for t, old in zip((c.k_pool, c.v_pool, c.kidx_pool, c.side_pool), before):
        assert torch.equal(t[:pc.first_spare].view(torch.int16), old)  # sources untouched
    written = torch.zeros((c.k_pool.shape[0], P), dtype=torch.bool, device=DEV)
    for s, want in enumerate(evict_ref(lens, mass, keep, sink, recent)):
        n = lens[s]
        assert b.kept[s].tolist() == want + [-1] * (keep - len(want))
        nl = 4 * len(want) - (-n) % 4
        assert int(b.new_lens[s]) == nl
        w = torch.tensor(want, dtype=torch.long, device=DEV)
        moved = b.mass[s, :len(want)]
        assert torch.equal(moved.nan_to_num(7.5), mass[s][w].nan_to_num(7.5))
        assert bool((b.mass[s, len(want):] == 0).all())
        t = torch.arange(nl, device=DEV)
        old = 4 * w[t // 4] + t % 4
        page, slot = pc.places(dst, s, nl, P)
        written[page, slot] = True
        assert torch.equal(c.k_pool[page, slot], pc.k[s][old])
        assert torch.equal(c.v_pool[page, slot], pc.v[s][old])
        assert torch.equal(c.kidx_pool[page, slot], pc.x[s][old])
        page, slot = pc.places(dst, s, nl // 4, P // 4)
        assert torch.equal(c.side_pool[page, slot], pc.side[s][w[:nl // 4]])
    # slots past the new lengths, and pages of nobody, stay as they were
    rest = c.k_pool[pc.first_spare:][~written[pc.first_spare:]]
    assert bool(rest.isnan().all())


def test_evict_flags():
    pc = Paged([400, 100], seed=2, spare=8)
    dst = torch.full((2, 7), -1, dtype=torch.int32, device=DEV)
    dst[0, 0] = pc.first_spare
    mass = torch.rand((2, 25), device=DEV)  # 25 blocks: the first sequence has 100
    b = qsa.alloc_evict(2, 25, 10)
    qsa.qsa_evict(pc.dims, pc.cache, pc.seq_lens, mass, 10, 0, 1, dst, b.kept, b.new_lens, b.mass)
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    # too long for its weights (16), no destination page (2)
    assert "flags=18" in str(e.value)
    assert b.new_lens.tolist() == [0, 40] and bool((b.kept[0] == -1).all())


# ------------------------------------------------------------ together

def test_serving_loop():
    """Norm + rotation, append, chunk attention, weights, eviction, then a decode
    step and a dense decode token on the evicted cache."""
    from tests.gpu_harness import bits
    import oracle
    lens, chunks, Hq, Hkv, D, P, di = [700, 333], [200, 333], 16, 2, 128, 64, 64
    pc = Paged([500, 1], Hq, Hkv, P, di, seed=21, spare=40, width=12)
    c, d = pc.cache, pc.dims
    free = list(range(pc.first_spare, pc.first_spare + 40))
    for s, n in enumerate(lens):
        for j in range(-(-n // P)):
            if int(c.block_table[s, j]) < 0:
                c.block_table[s, j] = free.pop()
    Nq = sum(chunks)
    seq = torch.cat([torch.full((T,), s) for s, T in enumerate(chunks)]).int().to(DEV)
    pos = torch.cat([torch.arange(n - T, n) for n, T in zip(lens, chunks)]).int().to(DEV)
    qkv = randn((Nq, Hq + 2 * Hkv, D), 3)
    ones = torch.ones(D, device=DEV)
    rope = qsa.rope_table(1024, 128)
    q = torch.empty((Nq, Hq, D), dtype=torch.bfloat16, device=DEV)
    k = torch.empty((Nq, Hkv, D), dtype=torch.bfloat16, device=DEV)
    qsa.qsa_qk_norm_rope(pos, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], ones, ones, 1e-6, rope, q, k)
    v = qkv[:, Hq + Hkv:].contiguous()
    x = randn((Nq, di), 4)
    qsa.qsa_append(d, c, seq, pos, k, v, x)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 200, 533], dtype=torch.int32, device=DEV)
    b = qsa.alloc_chunk_attention(d, 2, Nq, out_dtype=torch.float32)
    qsa.qsa_chunk_attention(d, c, seq_lens, start, q, b.out, b.lse, b.ws)
    ld = qsa.ld_for(lens)
    m = qsa.alloc_attention_mass(d, 2, Nq, ld)
    qsa.qsa_attention_mass(d, c, seq_lens, start, q, b.lse, None, m.mass, m.ws)
    # every row and head hands out one unit of weight
    assert abs(float(m.mass[0].sum()) / (200 * Hq) - 1) < 1e-3
    assert abs(float(m.mass[1].sum()) / (333 * Hq) - 1) < 1e-3
    # the append built the side keys of the chunk's blocks; the context's are made up
    pc.lens = lens
    pc.k = [torch.cat((pc.k[0], k[:200])), k[200:]]
    pc.v = [torch.cat((pc.v[0], v[:200])), v[200:]]
    pc.x = [torch.cat((pc.x[0], x[:200])), x[200:]]
    ref, lse, size, mass = attention_ref(pc, chunks, q)
    assert bool(((b.out.double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6).all())
    for s in range(2):
        assert bool(((m.mass[s, :mass[s].numel()] - mass[s]).abs() <= 2e-3 * mass[s] + 1e-6).all())

    keep = 60
    dst = torch.full((2, 12), -1, dtype=torch.int32, device=DEV)
    for s in range(2):
        for j in range(-(-(4 * keep + 4) // P)):
            dst[s, j] = free.pop()
    e = qsa.alloc_evict(2, ld, keep)
    qsa.qsa_evict(d, c, seq_lens, m.mass, keep, 1, 8, dst, e.kept, e.new_lens, e.mass, e.ws)
    small = qsa.QsaCache(c.k_pool, c.v_pool, c.kidx_pool, c.side_pool, dst)
    new = e.new_lens.tolist()
    assert new == [240, 237]
    # one more token per sequence: rotated at its true position, stored at its place
    q1, q_idx, w = randn((2, Hq, D), 7), randn((2, 4, di), 8), torch.rand((2, 4), device=DEV)
    kvx = randn((2, Hkv, D), 9), randn((2, Hkv, D), 10), randn((2, di), 11)
    now = (e.new_lens + 1).int()
    step = qsa.alloc_step(d, 2, ld, 32, 2)
    qsa.decode_step(d, small, now, q1, q_idx, w, 32, 2, step,
                    append=(torch.arange(2, dtype=torch.int32, device=DEV), e.new_lens, *kvx))
    dense = qsa.alloc_chunk_attention(d, 2, 2, out_dtype=torch.float32)
    qsa.qsa_chunk_attention(d, small, now, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV),
                            q1, dense.out, dense.lse, dense.ws)
    assert qsa.qsa_check_device_errors() == 0
    for s in range(2):
        kept = torch.tensor([j for j in e.kept[s].tolist() if j >= 0], device=DEV)
        t = torch.arange(new[s], device=DEV)
        old = 4 * kept[t // 4] + t % 4
        for a, one in zip((pc.k, pc.v, pc.x), kvx):
            a[s] = torch.cat((a[s][old], one[s:s + 1]))
        sel = step.sel[s].cpu().numpy()
        r = oracle.decode_sequence(bits(pc.x[s]), bits(pc.k[s]), bits(pc.v[s]), bits(q1[s]),
                                   bits(q_idx[s]), w[s].cpu().numpy(), new[s] + 1, 32, 2,
                                   d.scale, sel=sel)
        assert abs(step.out[s].float().cpu().numpy() - r["O"]).max() <= 1e-2
    pc.lens = [n + 1 for n in new]
    ref, lse, size, _ = attention_ref(pc, [1, 1], q1)
    assert bool(((dense.out.double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6).all())
    assert float((dense.lse.double() - lse).abs().max()) <= 1e-3


def test_captured_and_on_two_streams():
    """Captured and replayed on changed inputs, and two calls at once with a
    workspace each: the bits of plain calls."""
    pc = Paged([3001, 900], seed=31)
    start, q = pc.rows([70, 5], 1)
    start1, q1 = pc.rows([1, 1], 2)
    b, b1 = (qsa.alloc_chunk_attention(pc.dims, 2, n) for n in (75, 2))
    m = qsa.alloc_attention_mass(pc.dims, 2, 75, 751)
    e = qsa.alloc_evict(2, 751, 50)
    pos = torch.arange(75, dtype=torch.int32, device=DEV)
    rope = qsa.rope_table(100, 128)
    qr, raw = torch.empty_like(q), q.clone()
    P2 = Paged([3001, 900], seed=31, spare=16)
    dst = torch.full((2, 47), -1, dtype=torch.int32, device=DEV)
    dst[:, :4] = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4) + P2.first_spare

    def work(stream=None):
        qsa.qsa_qk_norm_rope(pos, raw, None, None, None, 0.0, rope, qr, stream=stream)
        qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, qr, b.out, b.lse, b.ws,
                                stream=stream)
        qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, qr, b.lse, None, m.mass, m.ws,
                               stream=stream)
        qsa.qsa_evict(P2.dims, P2.cache, P2.seq_lens, m.mass, 50, 1, 4, dst, e.kept, e.new_lens,
                      e.mass, e.ws, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (qr, b.out, b.lse, m.mass, e.kept, e.mass,
                                    P2.cache.k_pool[P2.first_spare:].view(torch.int16))]

    work()
    first = results()
    raw.copy_(raw.flip(0))
    work()
    second = results()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.capture_begin()
        work()
        g.capture_end()
    torch.cuda.synchronize()
    for want in (second, first):
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(results(), want))
        raw.copy_(raw.flip(0))
    # another stream at the same time, with its own buffers
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start1, q1, b1.out, b1.lse, b1.ws)
    torch.cuda.synchronize()
    alone = b1.out.clone()
    raw.copy_(raw.flip(0))
    raw.copy_(raw.flip(0))
    torch.cuda.synchronize()
    for _ in range(5):
        work(stream=side)
        qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start1, q1, b1.out, b1.lse, b1.ws)
    got = results()
    assert all(torch.equal(x, y) for x, y in zip(got, second))
    assert torch.equal(b1.out, alone)
    assert qsa.qsa_check_device_errors() == 0
