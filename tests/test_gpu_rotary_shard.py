"""GPU tests of the rotation of a query shard that begins inside a document: its rows count from the document's start."""
import pytest
import torch

import packed_sequence_flash_gb300 as psf
from test_gpu_cache import i32
from test_gpu_rotary import check, normal

pytestmark = pytest.mark.gpu

EDEVICE_ARGS = -4


@pytest.fixture(autouse=True)
def _clean_status():
    assert psf.device_status() == 0
    yield


def ids_of(rows):
    return torch.tensor([[d for d, n in row for _ in range(n)] for row in rows], dtype=torch.int32, device="cuda")


ROWS = {
    "one": [[(1, 40)]],
    "several": [[(1, 13), (2, 20), (3, 1), (4, 30)]],
    "padding": [[(1, 10), (0, 5), (2, 30), (0, 19)]],
    "batch": [[(1, 13), (2, 20), (3, 31)], [(4, 64)], [(5, 3), (6, 50), (0, 11)]],
}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("shard", [(0, 16), (7, 16), (16, 16), (21, 12), (30, 10)])
@pytest.mark.parametrize("skip_pad", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_rows_of_a_shard_are_those_of_the_whole(rows, shard, skip_pad, back):
    """Bit for bit what positions of the whole document give, for queries and for the keys that they see."""
    ids, (at, L) = ids_of(ROWS[rows]), shard
    B, S = ids.shape
    cu_q, cu_k, meta, _ = psf.build_doc_segments(ids, L, at, skip_pad=skip_pad)
    r = psf.Rotary(psf.rotary_frequencies(64), scale=0.75)
    call = psf.rotary_bwd if back else psf.rotary_fwd
    places = torch.tensor([[i for _, n in row for i in range(n)] for row in ROWS[rows]], dtype=torch.int32, device="cuda")
    real = ids > 0
    q, k = normal(B, 3, S, 64), normal(B, 2, S, 64, seed=1)
    want_q, want_k = call(q, k, r, positions=places)
    mine = q[:, :, at:at + L]
    got, none = call(mine, None, r, cu_seqlens=cu_q, dev_meta=meta, cu_seqlens_k=cu_k)
    assert none is None
    sel = real[:, at:at + L]
    assert torch.equal(got.transpose(1, 2)[sel], want_q[:, :, at:at + L].transpose(1, 2)[sel])
    got = call(None, k, r, cu_seqlens=cu_k, dev_meta=meta)[1]
    seen = real & (torch.arange(S, device="cuda") < at + L)
    assert torch.equal(got.transpose(1, 2)[seen], want_k.transpose(1, 2)[seen])
    if B == 1:  # packed rows, in place, the same numbers
        packed = mine[0].transpose(0, 1).contiguous()
        call(packed, None, r, None, cu_q, meta, packed, None, cu_k)
        assert torch.equal(packed[sel[0]], want_q[0, :, at:at + L].transpose(0, 1)[sel[0]])


@pytest.mark.parametrize("D,dim", [(128, 128), (72, 50)])
def test_alignment_against_64_bits(D, dim):
    """More rows than keys (negative places), as many, fewer, none of either; counts on the host and on the device."""
    cu_q, cu_k = [0, 5, 5, 12, 20, 30], [0, 2, 9, 16, 100, 100]
    inv = psf.rotary_frequencies(dim)
    pos = [i + n - m for s in range(5) for m, n in [(cu_q[s + 1] - cu_q[s], cu_k[s + 1] - cu_k[s])] for i in range(m)] + [0] * 3
    q, k = normal(33, 4, D), normal(33, 1, D, seed=1)
    r = psf.Rotary(inv)
    got = psf.rotary_fwd(q, k, r, cu_seqlens=i32(cu_q), cu_seqlens_k=i32(cu_k))
    check(q, k, inv, torch.tensor(pos), got)
    room = [i32(c + [10 ** 9] * 7) for c in (cu_q, cu_k)]
    again = psf.rotary_fwd(q, k, r, cu_seqlens=room[0], dev_meta=i32([5, 0, 0]), cu_seqlens_k=room[1])
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("cu_k", [[1, 5, 9], [0, 7, 5]])
def test_wrong_prefix_sums_are_reported(cu_k):
    q = normal(9, 1, 16)
    psf.rotary_fwd(q, None, psf.Rotary(psf.rotary_frequencies(16)), cu_seqlens=i32([0, 4, 9]), cu_seqlens_k=i32(cu_k))
    assert psf.device_status() == EDEVICE_ARGS


def test_arguments():
    q, r, cu = normal(9, 1, 16), psf.Rotary(psf.rotary_frequencies(16)), i32([0, 4, 9])
    for kw in (dict(cu_seqlens_k=cu), dict(cu_seqlens=cu, cu_seqlens_k=cu[:2]), dict(cu_seqlens=cu, cu_seqlens_k=cu.long()),
               dict(cu_seqlens=cu, cu_seqlens_k=cu, positions=i32([0] * 9))):
        with pytest.raises(ValueError):
            psf.rotary_fwd(q, None, r, **kw)


def test_a_sharded_step_is_the_whole_one():
    """Rotation, document attention and both backward calls by shards: outputs as the whole row's, dQ too, dK and dV as its sum."""
    ids = ids_of([[(1, 100), (2, 150), (0, 6)]])
    S, Hq, Hkv, D, scale = 256, 4, 2, 64, 0.125
    q, k, v, do = (normal(1, h, S, D, seed=s) for s, h in enumerate((Hq, Hkv, Hkv, Hq)))
    r = psf.Rotary(psf.rotary_frequencies(D))

    def step(at, L):
        mine = slice(at, at + L)
        cu_q, cu_k, meta, _ = psf.build_doc_segments(ids, L, at, skip_pad=True)
        kw_q, kw_k = dict(cu_seqlens=cu_q, dev_meta=meta, cu_seqlens_k=cu_k), dict(cu_seqlens=cu_k, dev_meta=meta)
        qr, kr = psf.rotary_fwd(q[:, :, mine], None, r, **kw_q)[0], psf.rotary_fwd(None, k, r, **kw_k)[1]
        out, lse, seg = psf.document_causal_attention(qr, kr, v, ids[:, mine].contiguous(), ids, at, scale)
        d = do[:, :, mine].contiguous()
        dq, dk, dv = psf.document_causal_attention_backward(d, qr, kr, v, out, lse, seg, scale)
        return out, psf.rotary_bwd(dq, None, r, **kw_q)[0], psf.rotary_bwd(None, dk, r, **kw_k)[1], dv

    whole = [x.double() for x in step(0, S)]
    parts = [step(at, 64) for at in range(0, S, 64)]
    cat = [torch.cat([p[i] for p in parts], 2).double() for i in (0, 1)] + [sum(p[i].double() for p in parts) for i in (2, 3)]
    for got, want in zip(cat, whole):  # (the attention's own bounds)
        assert float((got - want).norm() / want.norm()) <= 3e-2
    assert float((cat[0] - whole[0]).abs().max()) <= 2e-2
