"""Windowed attention over keys that are not finite.

A RoPE key belongs to one KV head: what it holds may change the outputs of that head's queries
only.  A score of -inf takes its token out of the softmax, +inf and NaN make the head's output
NaN, as the definition does; every other head is right within the bounds of test_gpu_window.py.
"""

import numpy as np
import pytest
import torch

from tests.helpers import assert_close
from tests.test_gpu_window import LAYERS, run_decode
from tests.window_helpers import Layer, hidden_tokens, make_cache, store

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# per sequence: (token, KV head, dims, value); tokens count from the end where negative
POISON = {
    "nan": [(-1, 1, slice(None), NAN), (-300, 0, slice(None), NAN), (0, 2, slice(0, 1), NAN)],
    "inf": [(-1, 0, slice(0, 1), INF), (-65, 1, slice(1, 2), -INF), (-300, 2, slice(3, 4), INF)],
    "sink_inf": [(0, 0, slice(0, 1), INF), (0, 1, slice(2, 3), -INF), (0, 2, slice(7, 8), -INF)],
}


def poisoned(layer, seq, what):
    """`seq` with non-finite keys (a copy), each in one KV head of one token."""
    s = dict(seq, kr=seq["kr"].clone())
    for t, g, dims, value in POISON[what]:
        t = t + seq["L"] if t < 0 else t
        if t >= 0:
            s["kr"][t, g % layer.n_kv, dims] = value
    return s


def check(got, ref, dtype, what):
    """Heads that the definition makes NaN are NaN throughout, the others are close."""
    bad = ~torch.isfinite(ref).all(-1)
    assert torch.isnan(got[bad]).all(), f"{what}: heads {bad.nonzero().flatten().tolist()} should be NaN"
    lost = ~torch.isfinite(got[~bad]).all(-1)
    assert not lost.any(), f"{what}: {int(lost.sum())} of {int((~bad).sum())} sound heads are not finite"
    if (~bad).any():
        assert_close(got[~bad].numpy(), ref[~bad].numpy(), dtype, what)


CASES = [("llama_dc64", 0), ("llama_dc256", 0), ("llama_int4", 0), ("llama_int2", 0), ("llama_r128", 0), ("smollm", 0),
         ("h24_gqa2", 0), ("h27_gqa3", 0), ("h32_gqa8_int2", 0), ("h20_dh40", 0), ("gqa64", 0), ("gqa64_int4", 0),
         ("llama_dc64", 3), ("smollm", 3), ("gqa64", 3), ("smollm", 1), ("tiny_f32", 0), ("tiny_f32", 1),
         ("gqa_f32_r3", 1)]


@pytest.mark.parametrize("what", list(POISON))
@pytest.mark.parametrize("name,kernel", CASES, ids=[f"{n}-{k}" for n, k in CASES])
def test_decode_window_keys(name, kernel, what):
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=21)
    lens = [1400, 700, 130, 1]
    B, T_cap = len(lens), 1408
    seqs = [layer.sequence(L) for L in lens]
    bad = [poisoned(layer, s, what) for s in seqs]
    q = layer.queries(B)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
    for n_sink, window in [(1, 1300), (1, 20), (3, 1405)]:
        cache = make_cache(mla, layer, B, T_cap, True)
        for b, s in enumerate(bad):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, n_sink, window))
        got = run_decode(mla, layer, cache, lens, q, n_sink, window, plan).double().cpu()
        for b, L in enumerate(lens):
            ref = layer.reference(q[b], bad[b], L - 1, n_sink, window)
            check(got[b], ref, layer.dtype, f"{name} {kernel} {what} sinks {n_sink} window {window} length {L}")
    plan.close()


CHUNK_CASES = [("llama_dc64", 0), ("llama_dc256", 0), ("llama_int4", 0), ("llama_int2", 0), ("smollm", 0), ("h24_gqa2", 0),
               ("h27_gqa3", 0), ("h32_gqa8_int2", 0), ("h20_dh40", 0), ("gqa64", 0), ("gqa64_int4", 0), ("llama_dc64", 3),
               ("smollm", 3), ("gqa64_int4", 3)]


@pytest.mark.parametrize("what", list(POISON))
@pytest.mark.parametrize("name,kernel", CHUNK_CASES, ids=[f"{n}-{k}" for n, k in CHUNK_CASES])
def test_chunk_window_keys(name, kernel, what):
    """The same for chunks, where some queries of a sequence see a key and others do not."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=22)
    lens, Q = [600, 330, 40], 37
    B, T_cap = len(lens), 640
    seqs = [layer.sequence(L) for L in lens]
    bad = [poisoned(layer, s, what) for s in seqs]
    q = layer.queries(B, Q)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
    for n_sink, window in [(1, 500), (1, 20), (3, 285)]:
        cache = make_cache(mla, layer, B, T_cap, n_sink == 3)
        for b, s in enumerate(bad):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - Q, n_sink, window))
        out = torch.full_like(q, 7.0, device="cuda")
        ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
        mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(),
                                    out, ws, n_sink, window)
        assert mla.mla_device_error(plan) == 0
        got = out.double().cpu()
        for b, L in enumerate(lens):
            for i in (0, 10, Q - 2, Q - 1):
                ref = layer.reference(q[b, i], bad[b], L - Q + i, n_sink, window)
                check(got[b, i], ref, "bf16", f"{name} {kernel} {what} sinks {n_sink} window {window} length {L} query {i}")
    plan.close()
