"""Refusals of the 8-bit cache and the tables that need no GPU: counts at the top of their 32
bits (before anything is launched; the pointers are never looked at), views of wrong types."""
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests.test_q8_host import FAKE, _append, lib

TOP = 2 ** 31 - 1


def tables(S, N):
    return lib().pa_build_tables(FAKE, 4, FAKE, FAKE, FAKE, S, FAKE, 8, FAKE, FAKE, 16, FAKE, FAKE, FAKE, N, None)


@pytest.mark.parametrize("count", [TOP, TOP - 31, TOP - 1022])
def test_counts_that_would_pass_32_bits_in_a_kernel_are_refused(count):
    assert tables(2, count) == P.PA_ERR_UNSUPPORTED
    assert tables(count, 9) == P.PA_ERR_UNSUPPORTED
    assert _append(N=count) == P.PA_ERR_UNSUPPORTED
    assert _append(S=count) == P.PA_ERR_UNSUPPORTED


def test_the_binding_refuses_counts_past_32_bits():
    i32 = torch.zeros(1, dtype=torch.int32)
    wide, cache = i32.expand(1, 2 ** 32 + 4), torch.zeros(2, P.pa_q8_block_bytes(2, 64, 16), dtype=torch.uint8)
    k = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="2.31"):
        P.pa_q8_append(k, k, cache, wide, i32, 16)
    with pytest.raises(ValueError, match="2.31"):
        P.pa_q8_decode(k, k, cache, wide, i32, 0.1, 2, 2, 64, 16)
    many = torch.zeros(1, 2, 64).expand(2 ** 31, 2, 64)
    with pytest.raises(ValueError, match="2.31"):
        P.pa_q8_append(many, many, cache, i32[None], i32, 16, query_start=i32.expand(2))
    args = dict(block_tables=i32[None], context_lens=i32, new_tokens=i32, free_list=i32, num_free=i32, block_size=16,
                slot_mapping=torch.zeros(3, dtype=torch.int64), query_start=i32.expand(2), granted=i32)
    for name, value in (("block_tables", wide), ("free_list", i32.expand(2 ** 31)),
                        ("slot_mapping", torch.zeros(1, dtype=torch.int64).expand(2 ** 32 + 7))):
        with pytest.raises(ValueError, match="2.31"):
            P.pa_build_tables(**{**args, name: value})


def test_views_of_a_cache_that_is_not_bytes_are_refused():
    size = P.pa_q8_block_bytes(2, 64, 16)
    for dtype in (torch.float32, torch.bfloat16, torch.int32):
        with pytest.raises(TypeError, match="uint8"):
            P.q8_views(torch.zeros(3, size, dtype=dtype), 2, 64, 16)
    cache = torch.zeros(3, size, dtype=torch.uint8)
    for same in (cache, cache.view(torch.int8), cache.view(torch.float8_e4m3fn)):
        assert P.q8_views(same, 2, 64, 16)[0].data_ptr() == cache.data_ptr()


def test_schedule_constants_have_one_value_in_every_file():
    """Device templates of pa_decode.cuh are instantiated in several files: a macro that one
    of them set otherwise would give one name two meanings."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(P.__file__), "csrc")
    files = {os.path.basename(f): open(f).read() for f in glob.glob(os.path.join(csrc, "*"))}
    for macro in ("PA_UNIT_COST", "PA_MIN_POSITIONS", "PA_STAGE_TOKENS"):
        assert [f for f, s in files.items() if re.search(rf"#define\s+{macro}\b", s)] == ["pa_internal.h"]
