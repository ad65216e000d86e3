"""The 8-bit decode gives the same answer every time, whichever part of a cut unit ends
last: nothing in it may depend on timing."""
import pytest
import torch

import paged_kv_cache_79_gb300 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def filled_cache(blocks, hkv, d, b, gen):
    """Random codes without NaN, scales of three neighbouring powers of two."""
    cache = P.alloc_q8_cache(blocks, hkv, d, b)
    codes, scales = P.q8_views(cache, hkv, d, b)
    codes.copy_((torch.randn(codes.shape, device=DEV, generator=gen) * 110).clamp_(-448, 448))
    scales.copy_(2.0 ** torch.randint(-8, -5, scales.shape, device=DEV, generator=gen))
    return cache


def cut_units(stages, fraction, d, b, hkv, gen):
    """A batch of `fraction` equal units per CTA of two per SM: the CTAs' equal shares end
    inside most of the units, and which part of one ends last changes from call to call.
    (cache, block tables, lengths)"""
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    seqs, tokens = max(1, int(ctas * fraction) // hkv), stages * 8192 // (2 * d)
    blocks = tokens // b
    cache = filled_cache(seqs * blocks, hkv, d, b, gen)
    bt = torch.randperm(seqs * blocks, device=DEV, generator=gen).int().view(seqs, blocks)
    return cache, bt, tokens - torch.arange(seqs, device=DEV, dtype=torch.int32) % 5


def calls(q, cache, bt, cl, scale, hq, hkv, d, b, rounds):
    """Ten outputs at a time, from memory and from the L2 cache in turn."""
    ws = torch.zeros(P.pa_q8_decode_workspace_size(len(cl), hq, hkv, d, b, bt.shape[1]), dtype=torch.uint8, device=DEV)
    flush = torch.zeros(64 << 20, dtype=torch.float32, device=DEV)
    outs = [torch.empty_like(q) for _ in range(10)]
    for rep in range(rounds):
        if rep % 2:
            flush.add_(1.0)
        for out in outs:
            P.pa_q8_decode(out, q, cache, bt, cl, scale, hq, hkv, d, b, workspace=ws)
        yield outs


@pytest.mark.parametrize("dtype,value", [("f32", 2.0 ** 126), ("bf16", 2.0 ** 126), ("f16", float("inf"))])
@pytest.mark.parametrize("d,b,hq,hkv,stages,fraction", [(128, 16, 16, 8, 500, 0.5), (64, 32, 8, 8, 26, 0.5)])
def test_rows_whose_scores_all_overflow_are_zero(dtype, value, d, b, hq, hkv, stages, fraction):
    """Every score of some rows is -inf: nothing has weight, in either part of a cut unit."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    cache, bt, cl = cut_units(stages, fraction, d, b, hkv, gen)
    codes, scales = P.q8_views(cache, hkv, d, b)
    codes[:, :, 0] = torch.full((), 64.0, device=DEV).to(codes.dtype)
    scales[:, :, 0] = 1.0
    q = torch.randn(len(cl), hq, d, device=DEV, generator=gen).to(TD[dtype])
    q[:, ::2] = value
    for outs in calls(q, cache, bt, cl, -1.0, hq, hkv, d, b, 6):
        for out in outs:
            assert not out[:, ::2].any() and torch.isfinite(out[:, 1::2].float()).all()
    assert P.pa_device_errors() == 0


@pytest.mark.parametrize("dtype,value", [("f32", 2.0 ** 126), ("bf16", 2.0 ** 126)])
@pytest.mark.parametrize("hq,tokens", [(16, 60000), (4, 60000), (1, 60000), (16, 6000), (5, 1500)])
def test_overflowing_rows_of_one_unit_in_many_parts(dtype, value, hq, tokens):
    """The same for a single unit over all CTAs, more parts than fit the merge's room too."""
    d, b = 64, 16
    gen = torch.Generator(device=DEV).manual_seed(5)
    cache = filled_cache(tokens // b + 1, 1, d, b, gen)
    codes, scales = P.q8_views(cache, 1, d, b)
    codes[:, :, 0] = torch.full((), 64.0, device=DEV).to(codes.dtype)
    scales[:, :, 0] = 1.0
    bt = torch.randperm(len(cache), device=DEV, generator=gen).int()[None]
    cl = torch.tensor([tokens], dtype=torch.int32, device=DEV)
    q = torch.randn(1, hq, d, device=DEV, generator=gen).to(TD[dtype])
    q[:, ::2] = value
    out = torch.empty_like(q)
    P.pa_q8_decode(out, q, cache, bt, cl, -1.0, hq, 1, d, b)
    assert not out[:, ::2].any() and torch.isfinite(out[:, 1::2].float()).all()


@pytest.mark.parametrize("dtype,d,b,hq,hkv,stages,fraction", [
    ("f32", 128, 16, 64, 8, 600, 0.5),         # two CTAs' shares per unit, both the same length
    ("f32", 128, 32, 16, 8, 500, 0.7),         # cuts at every place of a unit
    ("f32", 64, 16, 32, 8, 400, 0.6),
    ("f32", 128, 16, 8, 8, 26, 0.5),           # short parts that end within a microsecond
    ("f32", 128, 16, 96, 8, 500, 0.5),         # 12 rows per unit
    ("bf16", 128, 16, 16, 8, 30, 0.6),
    ("f16", 64, 32, 26, 2, 20, 0.7),           # 13 rows per unit
])
def test_units_cut_once_repeat_bit_for_bit(dtype, d, b, hq, hkv, stages, fraction):
    gen = torch.Generator(device=DEV).manual_seed(3)
    cache, bt, cl = cut_units(stages, fraction, d, b, hkv, gen)
    q = torch.randn(len(cl), hq, d, device=DEV, generator=gen).to(TD[dtype])
    first = None
    for outs in calls(q, cache, bt, cl, 0.1, hq, hkv, d, b, 20):
        if first is None:
            first = outs[0].clone()
        for out in outs:
            assert torch.equal(out, first), f"{(out != first).sum().item()} of {out.numel()} values differ"
    assert torch.isfinite(first.float()).all()
    assert P.pa_device_errors() == 0
