"""The dense-path calls at the ends of their ranges: many sequences, long
contexts, unusual scales, queries whose weights do not belong to the LSEs given,
weights that do not fit the eviction's shared memory, workspaces that two
captured calls share in order. Tolerances as in test_gpu_dense.py."""

from __future__ import annotations

import dataclasses
import math

import pytest
import torch

from block_sparse_decode_b200 import qsa
from tests.test_gpu_dense import DEV, HALF, Paged, attention_ref, evict_ref, randn

pytestmark = pytest.mark.gpu


def attend(pc, start, q, out_dtype=torch.float32):
    b = qsa.alloc_chunk_attention(pc.dims, len(pc.lens), q.shape[0], out_dtype=out_dtype)
    b.ws.random_(0, 255)
    qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    return b


def weigh(pc, start, q, lse, ld=None):
    m = qsa.alloc_attention_mass(pc.dims, len(pc.lens), q.shape[0], ld or qsa.ld_for(pc.lens))
    m.ws.random_(0, 255)
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse, None, m.mass, m.ws)
    assert qsa.qsa_check_device_errors() == 0
    return m.mass


def check(pc, chunks, q, b, mass=None):
    ref, lse, size, w = attention_ref(pc, chunks, q)
    assert bool(((b.out.double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6).all())
    assert float((b.lse.double() - lse).abs().max()) <= 1e-3
    if mass is not None:
        for s, want in enumerate(w):
            got = mass[s, :want.numel()].double()
            assert bool(((got - want).abs() <= 1e-3 * want + 1e-6).all())
            assert bool((mass[s, want.numel():] == 0).all())


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-3, 0.5])
def test_scales(scale):
    pc = Paged([400, 131], 8, 2, 32, seed=5)
    pc.dims = qsa.QsaDims(8, 2, 128, 4, 64, 32, scale)
    start, q = pc.rows([37, 131], 6)
    b = attend(pc, start, q)
    check(pc, [37, 131], q, b, weigh(pc, start, q, b.lse))


@pytest.mark.parametrize("S,longest,T,Hq,Hkv", [(1300, 90, 1, 8, 2), (1200, 40, 3, 4, 4)])
def test_many_sequences(S, longest, T, Hq, Hkv):
    """More sequences (and groups) than the plan has threads; some have no rows."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(T, longest, (S,), generator=g).tolist()
    chunks = torch.randint(0, T + 1, (S,), generator=g).tolist()
    pc = Paged(lens, Hq, Hkv, 16, seed=S)
    start, q = pc.rows(chunks, 7)
    b = attend(pc, start, q)
    check(pc, chunks, q, b, weigh(pc, start, q, b.lse))


@pytest.mark.parametrize("lens,chunks,P", [([70001], [1], 64), ([33000, 5], [9, 5], 1024),
                                           ([8200, 130], [700, 130], 12)])
def test_long_contexts(lens, chunks, P):
    pc = Paged(lens, 8, 1, P, seed=11, scale=2.0)
    start, q = pc.rows(chunks, 8)
    b = attend(pc, start, q)
    check(pc, chunks, q, b, weigh(pc, start, q, b.lse))


def test_long_items():
    """Items of 2^19 key tiles, longer than any wait for one tile may last. Every
    page of a sequence is the same one, so its LSE is that page's, plus ln(pages).
    A row's sum adds 2^19 partial sums in fp32, split over two halves of the tile
    and over blocks: each addition is off by 2^-24 of the sum, 2^-5 in all."""
    P, L, S = 1024, 2 ** 26, 160
    pc = Paged([P], 8, 1, P, seed=21)
    start, q = pc.rows([1], 9)
    near = attend(pc, start, q)
    table = torch.full((S, L // P), int(pc.cache.block_table[0, 0]), dtype=torch.int32, device=DEV)
    cache = dataclasses.replace(pc.cache, block_table=table)
    lens = torch.full((S,), L, dtype=torch.int32, device=DEV)
    row_start = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    b = qsa.alloc_chunk_attention(pc.dims, S, S, out_dtype=torch.float32)
    qsa.qsa_chunk_attention(pc.dims, cache, lens, row_start, q.expand(S, -1, -1).contiguous(),
                            b.out, b.lse, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    want = near.lse.double() + math.log(L // P)
    assert float((b.lse.double() - want).abs().max()) <= 2.0 ** -5 + 1e-3
    assert bool(torch.isfinite(b.out).all())


@pytest.mark.parametrize("longest,T", [(128, 1), (256, 1), (128, 40)])
def test_short_items_repeat(longest, T):
    """Items of one or two steps, one behind the other in every CTA: an item's
    sums take the place of its last maxima, and the next item's maxima theirs.
    The results are right, and the same bits call after call."""
    g = torch.Generator().manual_seed(longest + T)
    S = 600
    lens = torch.randint(T, longest + 1, (S,), generator=g).tolist()
    pc = Paged(lens, 32, 4, 64, seed=40, scale=2.0)
    start, q = pc.rows([T] * S, 12, 1.5)
    b = attend(pc, start, q)
    few = 24  # (the sequences with a reference)
    part = Paged(lens[:few], 32, 4, 64, seed=40, scale=2.0)
    check(part, [T] * few, q[:few * T],
          qsa.ChunkBuffers(b.out[:few * T], b.lse[:few * T], b.ws))
    out, lse = b.out.clone(), b.lse.clone()
    for _ in range(20):
        b.out.fill_(math.nan)
        qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
    assert qsa.qsa_check_device_errors() == 0


@pytest.mark.parametrize("L,Hq", [(2 ** 28 + 2 ** 17 + 5, 8), (2 ** 30, 8), (2 ** 30, 5)])
def test_mass_far_before_the_chunk(L, Hq):
    """Tokens more than 2^28 before the rows, up to the longest sequence there may
    be. The queries are zero, so every weight of row i is 1 / (the tokens it sees).
    Every page of the sequence is the same one. The LSE is rounded to 24 bits, off
    by at most 2^-20 (it is below 32: half a step of 2^-19), and scaled by log2(e):
    as much again. With the exponential's and the sums' roundings 2^-17 holds all."""
    P, T = 1024, 3
    pc = Paged([P], Hq, 1, P, seed=22)
    pages = -(-L // P)
    table = pc.cache.block_table[:1, :1].expand(1, pages).contiguous()
    cache = dataclasses.replace(pc.cache, block_table=table)
    q = torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    sees = [L - T + i + 1 for i in range(T)]
    lse = torch.tensor(sees, dtype=torch.float64, device=DEV).log().float()[:, None]
    lse = lse.expand(T, Hq).contiguous()
    m = qsa.alloc_attention_mass(pc.dims, 1, T, -(-L // 4))
    qsa.qsa_attention_mass(pc.dims, cache, lens, start, q, lse, None, m.mass, m.ws)
    assert qsa.qsa_check_device_errors() == 0
    whole = (L - T) // 4  # blocks that every row sees
    want = 4 * Hq * sum(1 / n for n in sees)
    assert float((m.mass[0, :whole] - want).abs().max()) <= 2.0 ** -17 * want
    for j in range(whole, -(-L // 4)):
        want = Hq * sum(max(0, min(4, n - 4 * j)) / n for n in sees)
        assert abs(float(m.mass[0, j]) - want) <= 2.0 ** -17 * want


@pytest.mark.parametrize("L,T,S,Hq,flat", [
    (128 * 1025, 1, 150, 8, True), (128 * 1025 + 1, 1, 300, 8, False), (2 ** 18 + 1, 1, 400, 5, True),
    (2 ** 18 + 77, 33, 90, 8, False), (128 * 2050 + 9, 32, 200, 8, True), (2 ** 22 + 130, 1, 160, 8, True),
    (2 ** 22 + 130, 1, 1, 8, False), (2 ** 24 + 3, 20, 10, 6, True), (2 ** 26, 1, 160, 8, True)])
def test_long_sums(L, T, S, Hq, flat):
    """Items of many steps, whole and shared, of one and of two tiles: results and
    LSEs as exact as those of short ones. The values are positive, so that what
    the additions lose adds up too; every page of a sequence is the same one.
    A part of 1,024 steps makes up to 8 * 1,025 additions in the tensor cores, off
    by at most 2^-23 of the sum each: 2^-10 + 2^-12 in all, next to the bound that
    every result has. With equal scores (flat) every weight is 1 and none is
    rounded. The row sums add 2^10 values a part and up to 2^9 parts in fp32,
    2^-24 each: 2^-13; and the LSE is held to 2^-20."""
    P = 1024
    pc = Paged([P], Hq, 1, P, seed=26)
    pc.v[0] = pc.v[0].abs() + 0.25
    page, slot = pc.places(pc.cache.block_table, 0, P, P)
    pc.cache.v_pool[page, slot] = pc.v[0]
    pages = -(-L // P)
    table = pc.cache.block_table[:1, :1].expand(S, pages).contiguous()
    cache = dataclasses.replace(pc.cache, block_table=table)
    q = randn((S * T, Hq, 128), 18) * (0.0 if flat else 1.0)
    start = torch.arange(S + 1, dtype=torch.int32, device=DEV) * T
    lens = torch.full((S,), L, dtype=torch.int32, device=DEV)
    b = qsa.alloc_chunk_attention(pc.dims, S, S * T, out_dtype=torch.float32)
    b.ws.random_(0, 255)
    qsa.qsa_chunk_attention(pc.dims, cache, lens, start, q, b.out, b.lse, b.ws)
    assert qsa.qsa_check_device_errors() == 0
    # how often a row sees each token of the page
    sees = (L - T + 1 + torch.arange(T, device=DEV)).repeat(S)
    n = (sees[:, None] - torch.arange(P, device=DEV) + P - 1) // P
    z = torch.einsum("rhd,td->rht", q.double(), pc.k[0][:, 0].double()) * pc.dims.scale
    z = z + n.double().log()[:, None]
    lse = torch.logsumexp(z, -1)
    ref = torch.einsum("rht,td->rhd", torch.exp(z - lse[..., None]), pc.v[0][:, 0].double())
    bound = 2.0 ** -10 + 2.0 ** -12 + (0.0 if flat else HALF + 2.0 ** -12)
    assert bool(((b.out.double() - ref).abs() <= bound * ref).all())
    bound = 2.0 ** -13 + 2.0 ** -19 + (0.0 if flat else 1e-3)
    assert float((b.lse.double() - lse).abs().max()) <= bound
    again = qsa.alloc_chunk_attention(pc.dims, S, S * T, out_dtype=torch.bfloat16)
    qsa.qsa_chunk_attention(pc.dims, cache, lens, start, q, again.out, again.lse, b.ws)
    assert torch.equal(again.out, b.out.to(torch.bfloat16)) and torch.equal(again.lse, b.lse)


def test_more_work_than_a_block_can_count():
    """65,535 rows of 16 KV heads over 2^30 tokens: past 2^30 units of work per block
    of the grid (5 * 10^11 over some 150), so the call is flagged and writes nothing."""
    P, L, T = 1024, 2 ** 30, 65535
    pc = Paged([P], 128, 16, P, seed=25)
    table = pc.cache.block_table[:1, :1].expand(1, L // P).contiguous()
    cache = dataclasses.replace(pc.cache, block_table=table)
    q = torch.zeros((T, 128, 128), dtype=torch.bfloat16, device=DEV)
    b = qsa.alloc_chunk_attention(pc.dims, 1, T)
    b.out.fill_(5.0), b.lse.fill_(5.0), b.ws.zero_()
    qsa.qsa_chunk_attention(pc.dims, cache, torch.tensor([L], dtype=torch.int32, device=DEV),
                            torch.tensor([0, T], dtype=torch.int32, device=DEV), q, b.out, b.lse,
                            b.ws)
    with pytest.raises(qsa.QsaError, match="flags=16"):
        qsa.qsa_check_device_errors()
    assert bool((b.out == 5).all()) and bool((b.lse == 5).all())


@pytest.mark.parametrize("lens,chunks,Hq,Hkv,P", [
    ([4099, 1500], [1, 1], 8, 2, 64), ([1000, 33, 257], [17, 16, 257], 32, 4, 48),
    ([700], [129], 21, 3, 4), ([5000], [1300], 8, 1, 64), ([30000, 7], [40, 7], 6, 1, 128)])
def test_mass_to_fp32(lens, chunks, Hq, Hkv, P):
    """Queries of -1, 0, 1 and keys of whole numbers up to 2: every score is exact, so
    what is left is the fp32 arithmetic on it. In the exponent of a weight, in
    units of log2 with scores below 8 and LSEs below 16: log2(e) in both
    products 2^-21 + 2^-20, the LSE's own rounding 2^-20, the two results' 2^-21
    + 2^-20, below 2^-18 in all; the exponential 2^-22; 32 columns added up four
    times in parallel 2^-19, and the rest of the sum 2^-21. Below 2^-17 together,
    with the sum of positive terms."""
    pc = Paged(lens, Hq, Hkv, P, seed=27)
    pc.dims = dataclasses.replace(pc.dims, scale=0.125)
    start, q = pc.rows(chunks, 19)
    q = q.clamp(-1, 1).round()
    for s, n in enumerate(lens):
        pc.k[s] = pc.k[s].clamp(-2, 2).round()
        page, slot = pc.places(pc.cache.block_table, s, n, P)
        pc.cache.k_pool[page, slot] = pc.k[s]
    _, lse, _, mass = attention_ref(pc, chunks, q)
    assert float(lse.max()) < 16
    got = weigh(pc, start, q, lse.float().contiguous())
    for s, want in enumerate(mass):
        assert bool(((got[s, :want.numel()].double() - want).abs() <= 2.0 ** -17 * want).all())


def test_mass_of_long_items():
    """Items of 262,144 steps (64 KV heads x 4,096 query blocks; 0.36 s), several in
    each block of the grid: longer than any wait for one step may last. The queries
    are zero, so a row's weights are 1 / (the tokens it sees). Tolerance as above."""
    P, L, T, Hkv = 1024, 3 * 2 ** 16, 65535, 64
    Hq = 8 * Hkv
    pc = Paged([P], Hq, Hkv, P, seed=24)
    table = pc.cache.block_table[:1, :1].expand(1, L // P).contiguous()
    cache = dataclasses.replace(pc.cache, block_table=table)
    q = torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device=DEV)
    sees = torch.arange(L - T + 1, L + 1, dtype=torch.float64, device=DEV)
    lse = sees.log().float()[:, None].expand(T, Hq).contiguous()
    m = qsa.alloc_attention_mass(pc.dims, 1, T, L // 4)
    qsa.qsa_attention_mass(pc.dims, cache, torch.tensor([L], dtype=torch.int32, device=DEV),
                           torch.tensor([0, T], dtype=torch.int32, device=DEV), q, lse, None,
                           m.mass, m.ws)
    assert qsa.qsa_check_device_errors() == 0
    # token t is seen by the rows that see more than t tokens
    rest = (1 / sees).flip(0).cumsum(0).flip(0)
    want = Hq * torch.cat((rest[:1].expand(L - T + 1), rest[1:])).view(-1, 4).sum(1)
    assert bool(((m.mass[0].double() - want).abs() <= 2.0 ** -17 * want).all())


def test_mass_without_rows():
    """No rows at all: mass is mass_in (or zeros, or itself), and a chunk that
    reaches past the rows is still flagged."""
    pc = Paged([100, 40], 8, 2, 64, seed=23)
    start, q = pc.rows([0, 0], 1)
    assert q.shape[0] == 0
    m = qsa.alloc_attention_mass(pc.dims, 2, 0, 25)
    lse = torch.empty((0, 8), device=DEV)
    base = torch.rand((2, 25), device=DEV)
    for given, want in ((base, base), (None, torch.zeros_like(base))):
        m.mass.fill_(math.nan)
        qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse, given, m.mass, m.ws)
        assert torch.equal(m.mass, want)
    again = base.clone()
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse, again, again, m.ws)
    assert torch.equal(again, base) and qsa.qsa_check_device_errors() == 0
    start[2] = 1
    qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, lse, base, m.mass, m.ws)
    with pytest.raises(qsa.QsaError, match="flags=16"):
        qsa.qsa_check_device_errors()
    assert torch.equal(m.mass, base)


def test_rows_of_chunks_add_up():
    """The rows of one call, and the same rows in calls of one token each, give
    the same results (each row of its own causal prefix)."""
    L, T = 300, 40
    pc = Paged([L], 16, 2, 64, seed=12)
    start, q = pc.rows([T], 9)
    whole = attend(pc, start, q)
    mass = weigh(pc, start, q, whole.lse, 75)
    total = torch.zeros_like(mass)
    for i in range(T):
        pc.lens = [L - T + i + 1]
        pc.seq_lens = torch.tensor(pc.lens, dtype=torch.int32, device=DEV)
        one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        b = attend(pc, one, q[i:i + 1].contiguous())
        # both are within the rounding of the weights of the exact result
        assert float((b.out[0] - whole.out[i]).abs().max()) <= 2 * HALF * 4
        assert float((b.lse[0] - whole.lse[i]).abs().max()) <= 1e-4
        total += weigh(pc, one, q[i:i + 1].contiguous(), b.lse, 75)
    assert bool(((total - mass).abs() <= 1e-4 * mass + 1e-6).all())


def test_weights_of_other_lse():
    """An LSE that is -inf gives no weight, +inf gives none either, and one below
    the row's own (as over a selection of blocks) weights above 1, which the sum
    holds up to 2^127."""
    pc = Paged([200], 8, 2, 64, seed=13)
    start, q = pc.rows([4], 10)
    b = attend(pc, start, q)
    _, lse, _, _ = attention_ref(pc, [4], q)
    mine = lse.float().clone()
    mine[0] = -math.inf
    mine[1] = math.inf
    mine[2] -= 20.0
    mine[3] = -1000.0
    mine[3, 1:] = -math.inf
    got = weigh(pc, start, q, mine)
    assert not bool(got.isnan().any())
    # row 3, head 0 alone: every weight is past 2^127 and counts as large
    mine[:3] = -math.inf
    assert bool((weigh(pc, start, q, mine) >= 2.0 ** 127).all())
    mine[3] = -math.inf
    assert bool((weigh(pc, start, q, mine) == 0).all())
    mine[2] = lse[2].float() - 20.0
    want = torch.zeros(200, dtype=torch.float64, device=DEV)
    for h in range(8):
        z = q[2, h].double() @ pc.k[0][:199, h // 4].double().T * pc.dims.scale
        want[:199] += torch.exp(z - mine[2, h].double())
    want = want.view(50, 4).sum(1)
    assert bool(((weigh(pc, start, q, mine)[0].double() - want).abs() <= 1e-3 * want).all())


@pytest.mark.parametrize("Hq,Hkv,L,T", [(8, 2, 200, 70), (8, 1, 140, 40), (4, 4, 300, 260)])
def test_weights_past_the_range(Hq, Hkv, L, T):
    """An LSE of NaN makes the blocks NaN that its row sees, and weights past
    fp32's range make them infinite, whichever column of the products the row and
    head are and whatever is added afterwards; the other blocks keep their bits."""
    pc = Paged([L], Hq, Hkv, 64, seed=16)
    start, q = pc.rows([T], 17)
    lse = attend(pc, start, q).lse
    clean = weigh(pc, start, q, lse)[0]
    for i in range(0, T, 1 if T < 100 else 13):
        sees = (L - T + i) // 4 + 1  # blocks
        for h in range(Hq):
            for value in (math.nan, -500.0):
                mine = lse.clone()
                mine[i, h] = value
                got = weigh(pc, start, q, mine)[0]
                hit = got.isnan() if math.isnan(value) else got == math.inf
                assert bool(hit[:sees].all()), (i, h, value)
                assert torch.equal(got[sees:], clean[sees:])


def test_largest_weights():
    """One weight of 2^126.5 (finite) and of 2^128.5 (not) in any column."""
    pc = Paged([1], 8, 1, 64, seed=17)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device=DEV)
    for h in range(8):
        for e in (126.5, 128.5):
            lse = torch.full((1, 8), math.inf, device=DEV)
            lse[0, h] = -e * math.log(2.0)
            got = float(weigh(pc, start, q, lse)[0, 0])
            # the LSE is rounded to steps of 2^-17, and so is the exponent
            assert got == math.inf if e > 128 else abs(got / 2.0 ** e - 1) <= 2.0 ** -15


def test_queries_of_others_do_not_matter():
    """NaN and infinity in the rows of other chunks and behind the last one reach
    neither a row's result nor its sequence's weights."""
    pc = Paged([150, 90, 61], 32, 4, 64, seed=14)
    start, q = pc.rows([5, 3, 2], 11, extra=3)
    clean = attend(pc, start, q.clone())
    want = weigh(pc, start, q, clean.lse)
    q[5:8] = math.nan
    q[10:] = math.inf
    lse = clean.lse.clone()
    lse[5:8] = math.nan
    got = attend(pc, start, q)
    rows = [0, 1, 2, 3, 4, 8, 9]
    assert torch.equal(got.out[rows], clean.out[rows])
    assert torch.equal(got.lse[rows], clean.lse[rows])
    mass = weigh(pc, start, q, lse)
    assert torch.equal(mass[0], want[0]) and torch.equal(mass[2], want[2])


@pytest.mark.parametrize("lens,chunks,Hq,Hkv", [
    ([70001], [1], 8, 2), ([3000, 200], [1, 1], 32, 4), ([515, 70], [90, 70], 16, 4),
    ([5000], [40], 32, 4), ([130] * 300, [1] * 300, 8, 2), ([700], [257], 5, 1), ([20000], [33], 8, 1)])
def test_scores_that_are_not_finite(lens, chunks, Hq, Hkv):
    """A head of a row whose scores hold NaN or +infinity gets NaN, as its formula
    does, whoever works on that part of its tokens; a score of -infinity is a
    weight of 0. The other rows and heads keep their bits."""
    pc = Paged(lens, Hq, Hkv, 64, seed=41)
    start, q = pc.rows(chunks, 13)
    for s, (n, T) in enumerate(zip(lens, chunks)):
        pc.k[s][:, :, 0] = 0
        pc.k[s][(n - T) // 2, :, 0] = 2.0  # one token, seen by every row
        page, slot = pc.places(pc.cache.block_table, s, n, 64)
        pc.cache.k_pool[page, slot] = pc.k[s]
    rows = [int(start[s]) + T - 1 - T // 3 for s, T in enumerate(chunks)]
    q[rows, 3] = 0
    clean = attend(pc, start, q)
    q[rows, 0] = math.nan
    q[rows, 1, 5] = math.inf
    q[rows, 2] = 0
    q[rows, 2, 0] = 3e38  # 6e38 for the one token: past the scores' range
    q[rows, 3, 0] = -3e38
    got = attend(pc, start, q)
    bad = torch.zeros((q.shape[0], Hq), dtype=torch.bool, device=DEV)
    for h in range(3):
        bad[rows, h] = True
    assert bool(got.out[bad].isnan().all()) and bool(got.lse[bad].isnan().all())
    bad[rows, 3] = True
    assert torch.equal(got.out[~bad], clean.out[~bad])
    assert torch.equal(got.lse[~bad], clean.lse[~bad])
    ref, lse, size, _ = attention_ref(pc, chunks, q)  # (in 64 bits the score is finite)
    err = (got.out[rows, 3].double() - ref[rows, 3]).abs()
    assert bool((err <= (HALF + 2.0 ** -12) * size[rows, 3] + 1e-6).all())
    assert float((got.lse[rows, 3].double() - lse[rows, 3]).abs().max()) <= 1e-3


def test_scores_that_are_not_finite_in_long_items():
    """The same where an item is done in parts: a NaN that only the last tokens
    of the page bring reaches every part, a row of -infinity none."""
    P, L, S, Hq = 1024, 128 * 2050, 150, 8
    pc = Paged([P], Hq, 1, P, seed=43)
    pc.k[0][:, :, 0] = 0
    pc.k[0][P - 3, :, 0] = 2.0
    pc.k[0][:, :, 1] = 2.0
    page, slot = pc.places(pc.cache.block_table, 0, P, P)
    pc.cache.k_pool[page, slot] = pc.k[0]
    table = pc.cache.block_table[:1, :1].expand(S, -(-L // P)).contiguous()
    cache = dataclasses.replace(pc.cache, block_table=table)
    lens = torch.full((S,), L, dtype=torch.int32, device=DEV)
    start = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    q = randn((S, Hq, 128), 20)
    b = qsa.alloc_chunk_attention(pc.dims, S, S, out_dtype=torch.float32)

    def call():
        qsa.qsa_chunk_attention(pc.dims, cache, lens, start, q, b.out, b.lse, b.ws)
        assert qsa.qsa_check_device_errors() == 0
        return b.out.clone(), b.lse.clone()

    clean = call()
    q[::3, 0] = math.nan
    q[::3, 1] = 0
    q[::3, 1, 0] = 3e38
    q[::3, 2] = 0
    q[::3, 2, 1] = -3e38
    out, lse = call()
    assert bool(out[::3, :2].isnan().all()) and bool(lse[::3, :2].isnan().all())
    assert bool((out[::3, 2] == 0).all()) and bool((lse[::3, 2] == -math.inf).all())
    same = torch.ones((S, Hq), dtype=torch.bool, device=DEV)
    same[::3, :3] = False
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])


@pytest.mark.parametrize("lens,chunks", [([3000, 200], [1, 1]), ([515, 70], [90, 70]), ([70001], [1])])
def test_huge_scores(lens, chunks):
    """Scores up to 2^29 give weights; a row whose largest is beyond 2^30 (in units of
    log2) gets NaN and not, where the fp32 maximum was rounded up by 128 and more,
    zeros. What is far below the largest score has no weight, however far."""
    pc = Paged(lens, 8, 2, 64, seed=44)
    pc.dims = dataclasses.replace(pc.dims, scale=0.125)
    start, q = pc.rows(chunks, 21)
    for s, (n, T) in enumerate(zip(lens, chunks)):
        pc.k[s][:, :, :3] = 0
        pc.k[s][(n - T) // 2, :, 0] = 1.0  # one token, seen by every row
        pc.k[s][:, :, 1] = 1.0
        page, slot = pc.places(pc.cache.block_table, s, n, 64)
        pc.cache.k_pool[page, slot] = pc.k[s]
    rows = [int(start[s]) + T - 1 - T // 3 for s, T in enumerate(chunks)]
    q[rows] = 0
    held = ((0, 0, 2.0 ** 32), (1, 0, -2.0 ** 36), (2, 1, 2.0 ** 32), (3, 1, -2.0 ** 32))
    # (the first: the maximum is rounded up by 236; the second: down by 248)
    past = [(4, 0, 1.984375 * 2.0 ** 34), (5, 0, 1.40625 * 2.0 ** 34), (6, 1, -1.984375 * 2.0 ** 36),
            (7, 1, 1.8046875 * 2.0 ** 39)]
    for h, i, v in (*held, *past):
        q[rows, h, i] = v
    b = attend(pc, start, q)
    for h, _, _ in past:
        assert bool(b.out[rows, h].isnan().all()) and bool(b.lse[rows, h].isnan().all())
    ref, lse, size, _ = attention_ref(pc, chunks, q)
    mine = torch.ones((q.shape[0], 8), dtype=torch.bool, device=DEV)
    for h, _, _ in past:
        mine[rows, h] = False
    # Heads 2 and 3 have all scores equal, at 2^29: half a step of a part's LSE in
    # fp32 is 2^29 / 2^24 = 32, so the parts' weights against each other may be off
    # by e^32 either way, which leaves them any average of the values they see
    for s, n in enumerate(pc.lens):
        v = pc.v[s][:, :, None].float().expand(n, 2, 4, 128).reshape(n, 8, 128)[:, 2:4]
        o = b.out[rows[s], 2:4]
        slack = HALF * v.abs().amax(0)
        assert bool((o <= v.amax(0) + slack).all()) and bool((o >= v.amin(0) - slack).all())
    mine[rows, 2:4] = False
    assert bool(((b.out.double() - ref).abs() <= (HALF + 2.0 ** -12) * size + 1e-6)[mine].all())
    # (an LSE in fp32: half a step of it and of the maximum, once each more for log2)
    mine[rows, 2:4] = True
    err = (b.lse.double() - lse).abs()
    assert bool((err <= 1e-3 + 2.0 ** -22 * lse.abs())[mine].all())


def test_rows_without_any_weight():
    """All scores -infinity: no weight, as where nothing is seen."""
    pc = Paged([300, 70], 8, 2, 64, seed=42)
    for s, n in enumerate(pc.lens):
        pc.k[s][:, :, 0] = 2.0
        page, slot = pc.places(pc.cache.block_table, s, n, 64)
        pc.cache.k_pool[page, slot] = pc.k[s]
    start, q = pc.rows([1, 70], 14)
    q[:, ::2] = 0
    q[:, ::2, 0] = -3e38
    b = attend(pc, start, q)
    assert bool((b.out[:, ::2] == 0).all()) and bool((b.lse[:, ::2] == -math.inf).all())
    assert bool(torch.isfinite(b.lse[:, 1::2]).all())


@pytest.mark.parametrize("keep", [3, 40000])
def test_evict_long_sequences(keep):
    """More blocks than the selection keeps in shared memory, next to short ones."""
    lens = [4 * 60001 + 2, 17]
    P, Hkv = 256, 1
    per = -(-4 * keep // P)
    pc = Paged(lens, 4, Hkv, P, 64, seed=keep, spare=2 * per)
    ld = qsa.ld_for(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    mass = torch.randint(0, 5000, (2, ld), generator=g, device=DEV).float()
    width = pc.cache.block_table.shape[1]
    dst = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    dst[:, :per] = torch.arange(2 * per, dtype=torch.int32, device=DEV).view(2, per) + pc.first_spare
    b = qsa.alloc_evict(2, ld, keep)
    qsa.qsa_evict(pc.dims, pc.cache, pc.seq_lens, mass, keep, 1, 1, dst, b.kept, b.new_lens, b.mass)
    assert qsa.qsa_check_device_errors() == 0
    for s, want in enumerate(evict_ref(lens, mass, keep, 1, 1)):
        assert b.kept[s, :len(want)].tolist() == want
        w = torch.tensor(want, device=DEV)
        nl = int(b.new_lens[s])
        assert nl == 4 * len(want) - (-lens[s]) % 4
        t = torch.arange(nl, device=DEV)
        page, slot = pc.places(dst, s, nl, P)
        assert torch.equal(pc.cache.k_pool[page, slot], pc.k[s][4 * w[t // 4] + t % 4])


def test_evict_past_the_tables():
    """Blocks whose source lies behind the table's last column, or on a page that
    is none, are flagged and not copied; the others are."""
    pc = Paged([64, 40], 8, 2, 16, 64, seed=28, spare=8, width=4)
    lens = torch.tensor([80, 40], dtype=torch.int32, device=DEV)  # 80 > 4 pages of 16
    pc.cache.block_table[1, 1] = -7
    dst = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    dst[:, :3] = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3) + pc.first_spare
    mass = torch.arange(20, dtype=torch.float32, device=DEV).flip(0).repeat(2, 1).contiguous()
    b = qsa.alloc_evict(2, 20, 10)
    qsa.qsa_evict(pc.dims, pc.cache, lens, mass, 10, 0, 4, dst, b.kept, b.new_lens, b.mass)
    with pytest.raises(qsa.QsaError, match="flags=6"):
        qsa.qsa_check_device_errors()
    assert b.kept[0].tolist() == [0, 1, 2, 3, 4, 5, 16, 17, 18, 19]
    assert b.kept[1].tolist() == list(range(10)) and b.new_lens.tolist() == [40, 40]
    for s, tokens in ((0, range(24)), (1, [*range(16), *range(32, 40)])):
        t = torch.tensor(list(tokens), device=DEV)
        got = pc.cache.k_pool[dst[s].long()[t // 16], t % 16]
        assert torch.equal(got, pc.k[s][t])
    for s, tokens in ((0, range(24, 40)), (1, range(16, 32))):
        t = torch.tensor(list(tokens), device=DEV)
        assert bool(pc.cache.k_pool[dst[s].long()[t // 16], t % 16].isnan().all())


def test_one_workspace_in_turn():
    """Two captured calls that share a workspace and run one after the other,
    replayed in either order, and an eager call between them."""
    pc = Paged([900, 40], 32, 4, 64, seed=15)
    a_start, a_q = pc.rows([33, 40], 1)
    b_start, b_q = pc.rows([1, 1], 2)
    a = qsa.alloc_chunk_attention(pc.dims, 2, 73)
    b = qsa.alloc_chunk_attention(pc.dims, 2, 2)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws

    def call(start, q, buf):
        qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, buf.out, buf.lse, ws)

    call(a_start, a_q, a)
    call(b_start, b_q, b)
    torch.cuda.synchronize()
    want = a.out.clone(), b.out.clone()
    graphs = []
    for args in ((a_start, a_q, a), (b_start, b_q, b)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*args)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1, 0)):
        a.out.zero_(), b.out.zero_()
        for i in order:
            graphs[i].replay()
            call(b_start, b_q, b)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_norm_rope_zero_rows_and_repeats():
    """Rows of zeros stay zero (eps > 0); the same position twice, and position 0."""
    q = torch.zeros((5, 4, 128), dtype=torch.bfloat16, device=DEV)
    q[1:] = randn((4, 4, 128), 3)
    q[2] = q[1]
    pos = torch.tensor([9, 5, 5, 0, 5], dtype=torch.int32, device=DEV)
    w = torch.rand(128, device=DEV)
    out = torch.empty_like(q)
    qsa.qsa_qk_norm_rope(pos, q, None, w, None, 1e-6, qsa.rope_table(10, 64), out)
    assert bool((out[0] == 0).all()) and torch.equal(out[1], out[2])
    y = q[3].float() * torch.rsqrt(q[3].float().square().mean(-1, keepdim=True) + 1e-6) * w
    assert bool(((out[3].float() - y).abs() <= HALF * y.abs() + 1e-6).all())


def test_other_devices_are_refused(monkeypatch):
    """Tensors of a device that is not the current one: refused, not launched."""
    q = randn((1, 2, 64), 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: q.device.index + 1)
    with pytest.raises(ValueError, match="current device"):
        qsa.qsa_qk_norm_rope(torch.zeros(1, dtype=torch.int32, device=DEV), q, None, None, None,
                             0.0, None, torch.empty_like(q))
