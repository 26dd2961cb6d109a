"""Refusals of the dense-path calls (no GPU needed: the checks run on the host,
before any CUDA call), and the rotation table."""

import ctypes
import math

import pytest
import torch

from block_sparse_decode_b200 import build, qsa

BAD, UNS = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return qsa.lib()


DIMS = dict(Hq=32, Hkv=4, D=128, Hi=16, di=128, P=64, scale=0.1)


def dims(**kw):
    return qsa._Dims(*{**DIMS, **kw}.values())


def cache(k=16, table=16, num_seqs=4):
    return qsa._Cache(k, 16, 16, 16, table, num_seqs, 8, 8)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), BAD), (dict(Hq=0), BAD), (dict(Hk=-1), BAD), (dict(D=96), UNS),
    (dict(rot=24), UNS), (dict(rot=144), UNS), (dict(rot=-16), UNS), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(max_pos=0), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(rope=None), BAD), (dict(pos=None), BAD), (dict(k_out=None), BAD), (dict(q=24), BAD),
    (dict(q_stride=128), BAD), (dict(q_stride=4 * 128 + 4), BAD), (dict(k_stride=0), BAD),
    (dict(qw=8), BAD), (dict(q_out=32, q=32, q_stride=1024), BAD),
])
def test_norm_rope_refusals(L, change, status):
    a = dict(N=2, Hq=4, Hk=2, D=128, pos=16, q=16, q_stride=512, k=16, k_stride=256, qw=16, kw=16,
             eps=1e-6, rope=16, max_pos=8, rot=128, pairs=0, q_out=32, k_out=32, stream=None)
    assert L.qsa_qk_norm_rope(*{**a, **change}.values()) == status
    assert L.qsa_last_error().decode()


def test_norm_rope_of_nothing(L):
    assert L.qsa_qk_norm_rope(0, 4, 0, 64, None, None, 0, None, 0, None, None, 0.0, None, 0, 0, 0,
                              None, None, None) == qsa.QSA_OK


CHUNK = dict(dims=dims(), cache=cache(), S=2, lens=16, start=16, Nq=5, q=16)


def call(fn, a):
    a = dict(a)
    a["dims"], a["cache"] = ctypes.byref(a["dims"]), ctypes.byref(a["cache"])
    return fn(*a.values())


COMMON = [(dict(dims=dims(D=64)), UNS), (dict(dims=dims(Hkv=5)), BAD), (dict(dims=dims(P=6)), UNS),
          (dict(dims=dims(Hkv=2)), UNS), (dict(cache=cache(k=17)), BAD),
          (dict(cache=cache(table=None)), BAD), (dict(S=5), BAD), (dict(S=-1), BAD),
          (dict(Nq=-1), BAD), (dict(Nq=65536), BAD), (dict(lens=None), BAD), (dict(start=None), BAD),
          (dict(q=None), BAD), (dict(q=24), BAD)]


@pytest.mark.parametrize("change,status", COMMON + [(dict(out=None), BAD), (dict(out=8), BAD),
                                                    (dict(ws=8), BAD)])
def test_chunk_attention_refusals(L, change, status):
    a = dict(CHUNK, out=16, bf16=1, lse=None, ws=16, ws_bytes=1 << 40, stream=None)
    assert call(L.qsa_chunk_attention, {**a, **change}) == status
    assert L.qsa_last_error().decode()


@pytest.mark.parametrize("change,status", COMMON + [(dict(lse=None), BAD), (dict(mass=None), BAD),
                                                    (dict(ld=0), BAD), (dict(ws=8), BAD)])
def test_attention_mass_refusals(L, change, status):
    a = dict(CHUNK, lse=16, mass_in=None, mass=16, ld=64, ws=16, ws_bytes=1 << 40, stream=None)
    assert call(L.qsa_attention_mass, {**a, **change}) == status
    assert L.qsa_last_error().decode()


def test_workspaces_are_asked_for(L):
    d = qsa.QsaDims(*DIMS.values())
    need = qsa.qsa_chunk_attention_workspace_size(d, 2, 5)
    a = dict(CHUNK, out=16, bf16=1, lse=None, ws=16, ws_bytes=need - 1, stream=None)
    if need:
        assert call(L.qsa_chunk_attention, a) == BAD and b"workspace" in L.qsa_last_error()
    need = qsa.qsa_attention_mass_workspace_size(d, 2, 5)
    a = dict(CHUNK, lse=16, mass_in=None, mass=16, ld=64, ws=None, ws_bytes=need, stream=None)
    if need:
        assert call(L.qsa_attention_mass, a) == BAD and b"workspace" in L.qsa_last_error()
    for f in (L.qsa_chunk_attention_workspace_size, L.qsa_attention_mass_workspace_size):
        assert f(None, 2, 5) == 0 and f(ctypes.byref(dims()), 0, 5) == 0


def test_workspace_without_rows(L):
    """The mass copies mass_in where there are no rows; the scratch it then asks
    for is what its query says."""
    need = L.qsa_attention_mass_workspace_size(ctypes.byref(dims()), 2, 0)
    a = dict(CHUNK, lse=None, mass_in=None, mass=16, ld=64, ws=16, ws_bytes=0, stream=None)
    a.update(Nq=0, q=None)
    assert call(L.qsa_attention_mass, a) == BAD
    assert f"workspace 0 bytes < {need} needed" in L.qsa_last_error().decode()


@pytest.mark.parametrize("change", [
    dict(Hq=2, Hkv=4), dict(Hq=1, Hkv=3), dict(Hq=256, Hkv=1), dict(Hq=6, Hkv=4), dict(Hq=0),
    dict(Hkv=0), dict(Hkv=-1), dict(D=64), dict(P=6), dict(S=65536), dict(S=2 ** 31 - 1), dict(S=-1),
    dict(Nq=65536), dict(Nq=2 ** 31 - 1), dict(Nq=-1)])
def test_workspaces_of_refused_calls_are_empty(L, change):
    """Sizes and dims that the calls refuse need no scratch (and end no process)."""
    sizes = dict(S=2, Nq=5)
    sizes.update({k: v for k, v in change.items() if k in sizes})
    d = qsa._Dims(*{**DIMS, **{k: v for k, v in change.items() if k in DIMS}}.values())
    for f in (L.qsa_chunk_attention_workspace_size, L.qsa_attention_mass_workspace_size):
        assert f(ctypes.byref(d), sizes["S"], sizes["Nq"]) == 0


@pytest.mark.parametrize("change,status", [
    (dict(dims=dims(di=96)), UNS), (dict(cache=cache(k=None)), BAD), (dict(B=5), BAD),
    (dict(B=-1), BAD), (dict(ld=0), UNS), (dict(keep=0), UNS), (dict(sink=-1), BAD),
    (dict(recent=0), BAD), (dict(sink=5), BAD), (dict(lens=None), BAD), (dict(mass=None), BAD),
    (dict(dst=None), BAD), (dict(kept=None), BAD), (dict(new=None), BAD), (dict(mass_out=None), BAD),
    (dict(mass_out=32), BAD), (dict(new=16), BAD), (dict(dst=16), BAD),
])
def test_evict_refusals(L, change, status):
    a = dict(dims=dims(), cache=cache(), B=2, lens=16, mass=32, ld=64, keep=8, sink=4, recent=4,
             dst=48, kept=64, new=80, mass_out=96, ws=None, ws_bytes=0, stream=None)
    assert call(L.qsa_evict, {**a, **change}) == status
    assert L.qsa_last_error().decode()


@pytest.mark.parametrize("change", [dict(ld=2 ** 28 + 1), dict(keep=2 ** 28 + 1),
                                    dict(ld=2 ** 31 - 1), dict(keep=2 ** 31 - 1)])
def test_evict_sizes_past_the_indexes(L, change):
    a = dict(dims=dims(), cache=cache(), B=2, lens=16, mass=32, ld=64, keep=8, sink=4, recent=4,
             dst=48, kept=64, new=80, mass_out=96, ws=None, ws_bytes=0, stream=None)
    assert call(L.qsa_evict, {**a, **change}) == qsa.QSA_ERR_UNSUPPORTED
    assert L.qsa_last_error().decode()


def test_calls_on_nothing(L):
    a = dict(CHUNK, out=None, bf16=1, lse=None, ws=None, ws_bytes=0, stream=None)
    assert call(L.qsa_chunk_attention, {**a, "S": 0}) == qsa.QSA_OK
    assert call(L.qsa_chunk_attention, {**a, "Nq": 0}) == qsa.QSA_OK
    a = dict(CHUNK, lse=None, mass_in=None, mass=None, ld=64, ws=None, ws_bytes=0, stream=None)
    assert call(L.qsa_attention_mass, {**a, "S": 0}) == qsa.QSA_OK


def test_rope_table():
    t = qsa.rope_table(300, 64, 5e5, device="cpu")
    assert t.shape == (300, 64) and t.dtype == torch.float32
    for p, i in ((0, 0), (299, 31), (123, 7)):
        a = p * 5e5 ** (-2 * i / 64)
        assert abs(float(t[p, i]) - math.cos(a)) < 1e-7
        assert abs(float(t[p, 32 + i]) - math.sin(a)) < 1e-7
    u = qsa.rope_table(10, 4, inv_freq=[1.0, 0.5], device="cpu")
    assert abs(float(u[9, 1]) - math.cos(4.5)) < 1e-7
    with pytest.raises(ValueError):
        qsa.rope_table(10, 4, inv_freq=[1.0], device="cpu")


def test_binding_refusals():
    bf = torch.bfloat16
    q = torch.zeros((2, 3, 64), dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qsa_qk_norm_rope(torch.zeros(2, dtype=torch.int32), q, None, None, None, 0.0, None, q)
    d = qsa.QsaDims(*DIMS.values())
    with pytest.raises(ValueError, match="row_start"):
        qsa.qsa_chunk_attention(d, None, torch.zeros(2, dtype=torch.int32),
                                torch.zeros(2, dtype=torch.int32), q, q)
    with pytest.raises(ValueError, match="q must have"):
        qsa.qsa_attention_mass(d, None, torch.zeros(2, dtype=torch.int32),
                               torch.zeros(3, dtype=torch.int32), q, None, None, None)


class Elsewhere(torch.Tensor):
    """A tensor that says it is on device 1."""

    def get_device(self):
        return 1


def _calls():
    i32, bf = torch.int32, torch.bfloat16
    d = qsa.QsaDims(8, 2, 128, 4, 64, 16, 0.1)
    z = torch.zeros
    pools = dict(k_pool=z((4, 16, 2, 128), dtype=bf), v_pool=z((4, 16, 2, 128), dtype=bf),
                 kidx_pool=z((4, 16, 64), dtype=bf), side_pool=z((4, 4, 64), dtype=bf),
                 block_table=z((2, 4), dtype=i32))
    rows = dict(seq_lens=z(2, dtype=i32), row_start=z(3, dtype=i32), q=z((5, 8, 128), dtype=bf))
    ws = z(16, dtype=torch.uint8)
    return {
        "norm": (lambda a: qsa.qsa_qk_norm_rope(eps=0.0, **a),
                 dict(pos=z(5, dtype=i32), q=z((5, 8, 128), dtype=bf), k=z((5, 2, 128), dtype=bf),
                      q_weight=z(128), k_weight=z(128), rope=z((9, 64)),
                      q_out=z((5, 8, 128), dtype=bf), k_out=z((5, 2, 128), dtype=bf)), ()),
        "attend": (lambda a, c: qsa.qsa_chunk_attention(d, c, **a),
                   dict(rows, out=z((5, 8, 128)), lse=z((5, 8)), ws=ws), pools),
        "mass": (lambda a, c: qsa.qsa_attention_mass(d, c, **a),
                 dict(rows, lse=z((5, 8)), mass_in=z((2, 7)), mass=z((2, 7)), ws=ws), pools),
        "evict": (lambda a, c: qsa.qsa_evict(d, c, keep=3, sink=1, recent=1, **a),
                  dict(seq_lens=z(2, dtype=i32), mass=z((2, 7)), dst_table=z((2, 4), dtype=i32),
                       kept=z((2, 3), dtype=i32), new_lens=z(2, dtype=i32), mass_out=z((2, 7)),
                       ws=ws), pools),
    }


@pytest.mark.parametrize("op", ["norm", "attend", "mass", "evict"])
@pytest.mark.parametrize("stream", [None, 0])
def test_every_tensor_has_to_be_on_the_current_device(monkeypatch, op, stream):
    """Any one tensor of another device, pools and scratch among them: refused
    before anything is launched, on an explicit stream too."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    call, args, pools = _calls()[op]
    skip = () if op == "evict" else ("kidx_pool", "side_pool")  # (not read by the others)
    for name in [*args, *(n for n in pools if n not in skip)]:
        a, p = dict(args, stream=stream), dict(pools)
        where = a if name in a else p
        where[name] = where[name].as_subclass(Elsewhere)
        with pytest.raises(ValueError, match="current device"):
            call(a, qsa.QsaCache(**p)) if p else call(a)
