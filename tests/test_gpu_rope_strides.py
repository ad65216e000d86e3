"""pa_rope and pa_rope_append through the C ABI: strides of a single token, of several."""
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from paged_kv_cache_79_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("stride", [0, 1, -7, 1 << 40])
@pytest.mark.parametrize("append", [False, True])
def test_strides_of_one_token_are_not_looked_at(stride, append):
    hq, hkv, d, B = 3, 2, 64, 16
    q, k, v = (torch.randn(1, h, d, device=DEV).half() for h in (hq, hkv, hkv))
    pos = torch.tensor([7], dtype=torch.int32, device=DEV)
    freqs = P.rope_frequencies(d)[0].to(DEV)
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    P.pa_rope(q2, q, k2, k, pos, freqs)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    kc, vc = torch.zeros(2, 2, B, hkv, d, device=DEV, dtype=torch.half)
    slot = torch.tensor([21], dtype=torch.int64, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    lib = _lib.load()
    if append:
        st = lib.pa_rope_append(qo.data_ptr(), stride, q.data_ptr(), stride, k.data_ptr(), stride, v.data_ptr(), stride,
                                kc.data_ptr(), vc.data_ptr(), pos.data_ptr(), slot.data_ptr(), freqs.data_ptr(), 1, hq,
                                hkv, d, d, 0, 1.0, B, 2, P.PA_F16, stream)
        ko = kc[1, 5][None]
        assert torch.equal(vc[1, 5], v[0]) and int(kc.count_nonzero()) == int(k2.count_nonzero())
    else:
        st = lib.pa_rope(qo.data_ptr(), stride, q.data_ptr(), stride, ko.data_ptr(), stride, k.data_ptr(), stride,
                         pos.data_ptr(), freqs.data_ptr(), 1, hq, hkv, d, d, 0, 1.0, P.PA_F16, stream)
    assert st == P.PA_OK
    assert torch.equal(qo, q2) and torch.equal(ko, k2)


def test_strides_of_several_tokens_are():
    """(Refused before anything is enqueued.)"""
    lib = _lib.load()
    fake = 1 << 20
    for stride in (0, 191, 193, 196):
        assert lib.pa_rope(fake, 192, fake, stride, fake, 128, fake, 128, fake, fake, 2, 3, 2, 64, 64, 0, 1.0, P.PA_F16,
                           None) == P.PA_ERR_INVALID
