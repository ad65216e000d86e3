"""What pa_attend refuses (no GPU needed: validation fails before anything is enqueued)."""
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from paged_kv_cache_79_gb300 import _lib

FAKE = 1 << 20   # a 16-byte aligned non-null value; never dereferenced


def _attend(**kw):
    a = dict(out=FAKE, lse=None, q=FAKE, qs=512, k=FAKE, v=FAKE, bt=FAKE, W=4, cl=FAKE, qst=FAKE, S=2, N=5, NB=8,
             scale=0.1, causal=1, Hq=4, Hkv=2, D=128, B=16, dt=2, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return _lib.load().pa_attend(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=0), P.PA_OK), (dict(N=0), P.PA_OK),
    (dict(out=None), P.PA_ERR_INVALID), (dict(q=None), P.PA_ERR_INVALID), (dict(k=None), P.PA_ERR_INVALID),
    (dict(v=None), P.PA_ERR_INVALID), (dict(bt=None), P.PA_ERR_INVALID), (dict(cl=None), P.PA_ERR_INVALID),
    (dict(qst=None), P.PA_ERR_INVALID), (dict(S=-1), P.PA_ERR_INVALID), (dict(N=-1), P.PA_ERR_INVALID),
    (dict(out=FAKE + 8), P.PA_ERR_INVALID), (dict(q=FAKE + 2), P.PA_ERR_INVALID), (dict(k=FAKE + 4), P.PA_ERR_INVALID),
    (dict(v=FAKE + 8), P.PA_ERR_INVALID), (dict(bt=FAKE + 2), P.PA_ERR_INVALID), (dict(cl=FAKE + 1), P.PA_ERR_INVALID),
    (dict(qst=FAKE + 2), P.PA_ERR_INVALID), (dict(lse=FAKE + 2), P.PA_ERR_INVALID), (dict(W=0), P.PA_ERR_INVALID),
    (dict(NB=0), P.PA_ERR_INVALID), (dict(Hq=5), P.PA_ERR_INVALID), (dict(Hkv=0), P.PA_ERR_INVALID),
    (dict(qs=508), P.PA_ERR_INVALID), (dict(qs=516), P.PA_ERR_INVALID), (dict(qs=256), P.PA_ERR_INVALID),
    (dict(qs=-512), P.PA_ERR_INVALID), (dict(D=96), P.PA_ERR_UNSUPPORTED), (dict(B=8), P.PA_ERR_UNSUPPORTED),
    (dict(dt=5), P.PA_ERR_UNSUPPORTED), (dict(NB=1 << 27), P.PA_ERR_INVALID), (dict(W=1 << 27), P.PA_ERR_INVALID),
    (dict(Hq=65536, Hkv=2, qs=1 << 24), P.PA_ERR_UNSUPPORTED), (dict(S=0x7fffffff), P.PA_ERR_UNSUPPORTED),
    (dict(N=0x7fffffff), P.PA_ERR_UNSUPPORTED), (dict(qs=1 << 36), P.PA_ERR_UNSUPPORTED),
])
def test_validation(kw, want):
    assert _attend(**kw) == want


def test_workspace_size():
    lib = _lib.load()
    bad = (1 << 64) - 1
    assert lib.pa_attend_workspace_size(4, 3, 64) == bad and lib.pa_attend_workspace_size(4, 2, 96) == bad
    if torch.cuda.is_available():
        assert P.pa_attend_workspace_size(4, 2, 64) < P.pa_attend_workspace_size(4, 2, 128)


def test_binding_refuses():
    q = torch.zeros(3, 4, 64)
    c = torch.zeros(8, 16, 2, 64)
    bt, cl, qs = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = dict(out=q, q=q, k_cache=c, v_cache=c, block_tables=bt, context_lens=cl, query_start=qs, scale=1.0,
                num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16)
    for kw, err in ((dict(), ValueError), (dict(q=q.half()), TypeError), (dict(query_start=qs.long()), TypeError),
                    (dict(query_start=qs[:2]), ValueError), (dict(num_kv_heads=4), ValueError),
                    (dict(block_size=32), ValueError), (dict(q=q[:2]), ValueError), (dict(block_tables=cl), ValueError),
                    (dict(lse=q[..., 0].half()), TypeError), (dict(lse=q[:2, :, 0].contiguous()), ValueError)):
        with pytest.raises(err):
            P.pa_attend(**{**good, **kw})
