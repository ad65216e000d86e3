"""The prompt side of a serving step, run together as an engine runs it: tables grown on the GPU,
rotary append, attention of the chunks, forks with their block copies, then decode steps of the
samples; every step against a plain float64 model of the sequences' own keys and values."""
import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Model:
    """The sequences as plain lists of rotated keys and values in 64 bits."""

    def __init__(self):
        self.k, self.v = {}, {}

    def attend(self, key, q, scale, causal_from=None):
        """q [n, Hq, d] over sequence `key`; query i sees causal_from + i + 1 keys (None: all)."""
        k, v = torch.stack(self.k[key]), torch.stack(self.v[key])          # [T, Hkv, d]
        g = q.shape[1] // k.shape[1]
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        s = torch.einsum("nhd,thd->nht", q.double(), k) * scale
        if causal_from is not None:
            seen = torch.arange(k.shape[0], device=DEV) <= causal_from + torch.arange(q.shape[0], device=DEV)[:, None]
            s = s.masked_fill(~seen[:, None], -torch.inf)
        return torch.einsum("nht,thd->nhd", torch.softmax(s, -1), v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("graph", [False, True])
def test_prompts_samples_and_decode(dtype, graph):
    """Two prompts in two chunks each, four and three samples, twelve decode steps.

    The model holds the rows that the cache holds (rounded once to the type), so what is left
    are the attention's own roundings: judged at 2^-6 (bf16), 2^-9 (fp16) and 2^-14 (fp32) of
    max |v|: eight half steps of the type's (fp32: sums of 300 terms at 2^-24 and products at
    2^-21, thirty-two times over)."""
    B, Hq, Hkv, d, NB, W = 16, 8, 2, 64, 200, 40
    tol = {torch.float32: 2.0 ** -14, torch.float16: 2.0 ** -9, torch.bfloat16: 2.0 ** -6}[dtype]
    gen = torch.Generator(DEV).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=DEV)
    caches = torch.full((2, NB, B, Hkv, d), float("nan"), device=DEV, dtype=dtype)
    freqs, amp = P.rope_frequencies(d, scaling="yarn", factor=4.0, original_len=512)
    freqs = freqs.to(DEV)
    scale = d ** -0.5
    free, num_free = torch.arange(NB, **i32), torch.tensor([NB], **i32)
    extra = torch.zeros(NB, **i32)
    model = Model()
    rows = caches.flatten(1, 2)

    def chunk(tables, lens, new, keys):
        """Grow, rotate and append, attend: one chunk of every sequence."""
        S, N = len(new), sum(new) + 5
        slots = torch.empty(N, dtype=torch.int64, device=DEV)
        starts, granted = torch.empty(S + 1, **i32), torch.empty(S, **i32)
        old = lens.tolist()
        P.pa_build_tables(tables, lens, torch.tensor(new, **i32), free, num_free, B, slots, starts, granted)
        assert granted.tolist() == new
        qkv = torch.randn(N, (Hq + 2 * Hkv) * d, device=DEV, generator=gen).to(dtype)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        pos = torch.zeros(N, **i32)
        pos[:sum(new)] = torch.cat([torch.arange(o, o + n, **i32) for o, n in zip(old, new)])
        q_out = torch.empty(N, Hq, d, device=DEV, dtype=dtype)
        P.pa_rope_append(q_out, q, k, v, caches[0], caches[1], pos, slots, freqs, amplitude=amp)
        out = torch.zeros(N, Hq, d, device=DEV, dtype=dtype)
        P.pa_attend(out, q_out, caches[0], caches[1], tables, lens, starts, scale, Hq, Hkv, d, B, causal=True)
        at = 0
        for key, o, n in zip(keys, old, new):
            mine = slots[at:at + n]
            model.k.setdefault(key, []).extend(rows[0][mine].double())
            model.v.setdefault(key, []).extend(rows[1][mine].double())
            assert torch.equal(rows[1][mine], v[at:at + n])
            want = model.attend(key, q_out[at:at + n], scale, causal_from=o)
            err = (out[at:at + n].double() - want).abs().max().item()
            assert err <= tol * torch.stack(model.v[key]).abs().max().item(), (key, err)
            at += n
        assert P.pa_device_errors() == 0

    tables, lens = torch.full((2, W), -1, **i32), torch.zeros(2, **i32)
    chunk(tables, lens, [150, 37], ["a", "b"])
    chunk(tables, lens, [99, 64], ["a", "b"])

    # samples: four of the first prompt, three of the second
    parents = [0, 0, 1, 0, 1, 1, 0]
    C = len(parents)
    tables2, lens2 = torch.empty(C, W, **i32), torch.empty(C, **i32)
    pairs, granted = torch.empty(C, 2, **i32), torch.empty(C, **i32)
    P.pa_fork_tables(tables2, lens2, tables, lens, torch.tensor(parents, **i32), extra, free, num_free, B, pairs, granted)
    P.pa_copy_blocks(caches[0], caches[1], pairs)
    assert granted.tolist() == [1] * C
    for i, p in enumerate(parents):
        model.k[i], model.v[i] = list(model.k["ab"[p]]), list(model.v["ab"[p]])
    del model.k["a"], model.k["b"]

    # decode steps, the fixed-shape launches captured once where `graph`
    new = torch.ones(C, **i32)
    slots, starts = torch.empty(C, dtype=torch.int64, device=DEV), torch.empty(C + 1, **i32)
    qkv = torch.empty(C, (Hq + 2 * Hkv) * d, device=DEV, dtype=dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    q_out, out, out2 = (torch.empty(C, Hq, d, device=DEV, dtype=dtype) for _ in range(3))
    pos = torch.empty(C, **i32)
    ws = P.alloc_workspace(C, Hq, Hkv, d, B, W)
    ws2 = torch.empty(P.pa_attend_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device=DEV)

    def step():
        pos.copy_(lens2)
        P.pa_build_tables(tables2, lens2, new, free, num_free, B, slots, starts, granted)
        P.pa_rope_append(q_out, q, k, v, caches[0], caches[1], pos, slots, freqs, amplitude=amp)
        P.pa_decode(out, q_out, caches[0], caches[1], tables2, lens2, scale, Hq, Hkv, d, B, workspace=ws)
        P.pa_attend(out2, q_out, caches[0], caches[1], tables2, lens2, starts, scale, Hq, Hkv, d, B, causal=True,
                    workspace=ws2)

    g = None
    for t in range(12):
        qkv.copy_(torch.randn(qkv.shape, device=DEV, generator=gen))
        if graph and t == 1:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        if g is not None:
            g.replay()
        else:
            step()
        assert granted.tolist() == [1] * C
        for i in range(C):
            model.k[i].append(rows[0][slots[i]].double())
            model.v[i].append(rows[1][slots[i]].double())
            want = model.attend(i, q_out[i:i + 1], scale)[0]
            bound = tol * torch.stack(model.v[i]).abs().max().item()
            assert (out[i].double() - want).abs().max() <= bound
            assert (out2[i].double() - want).abs().max() <= bound

    # finished: every block comes back
    nothing = torch.empty(0, **i32)
    P.pa_fork_tables(torch.empty(0, W, **i32), nothing, tables2, lens2, nothing, extra, free, num_free, B,
                     torch.empty(0, 2, **i32), nothing)
    assert int(num_free) == NB and sorted(free.tolist()) == list(range(NB)) and not extra.any()
    assert P.pa_device_errors() == 0
