"""Waits of the dense kernels that run out, on a real GPU without a fault.

The environment variable QSA_DEBUG_STALL_DENSE=n makes the warp that loads K
tiles stop silently after n of them in every block. The other roles wait for
tiles that never come, give up after their limit (0.27 s), wait for the copies
and products that are in flight, and free the tensor memory: the call is
reported as timed out, and the context goes on."""

from __future__ import annotations

import pytest
import torch

from block_sparse_decode_b200 import qsa
from tests.test_gpu_dense import Paged

pytestmark = pytest.mark.gpu


def timed_out():
    with pytest.raises(qsa.QsaError) as e:
        qsa.qsa_check_device_errors()
    assert e.value.status == qsa.QSA_ERR_TIMEOUT and "flags=32" in str(e.value)
    assert qsa.qsa_check_device_errors() == 0  # read and cleared


@pytest.mark.parametrize("lens,chunks", [([40000, 517], [700, 1]), ([60000, 300], [1, 1])])
@pytest.mark.parametrize("tiles", [0, 1, 4])
def test_lost_tiles_are_reported(monkeypatch, lens, chunks, tiles):
    """None, one or some tiles arrive: items of two tiles and of one, shared and
    whole, with more or fewer copies and products in flight when it stops."""
    pc = Paged(lens, 32, 4, 64, seed=50)
    start, q = pc.rows(chunks, 51)
    b = qsa.alloc_chunk_attention(pc.dims, 2, q.shape[0])
    m = qsa.alloc_attention_mass(pc.dims, 2, q.shape[0], qsa.ld_for(lens))
    b.ws.zero_(), m.ws.zero_()

    def attend():
        qsa.qsa_chunk_attention(pc.dims, pc.cache, pc.seq_lens, start, q, b.out, b.lse, b.ws)

    def weigh():
        qsa.qsa_attention_mass(pc.dims, pc.cache, pc.seq_lens, start, q, want[1], None, m.mass,
                               m.ws)

    attend()
    want = b.out.clone(), b.lse.clone()
    weigh()
    mass = m.mass.clone()
    assert qsa.qsa_check_device_errors() == 0
    for call in (attend, weigh):
        monkeypatch.setenv("QSA_DEBUG_STALL_DENSE", str(tiles))
        call()
        timed_out()
        monkeypatch.delenv("QSA_DEBUG_STALL_DENSE")
        attend()
        weigh()
        assert qsa.qsa_check_device_errors() == 0
        assert torch.equal(b.out, want[0]) and torch.equal(b.lse, want[1])
        assert torch.equal(m.mass, mass)
