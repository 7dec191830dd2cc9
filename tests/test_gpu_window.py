"""Sliding-window attention with sinks (mla_decode_window, mla_decode_chunk_window) against the
definition in float64.

Hidden tokens hold NaN in every cache array, so a kernel that reads one shows it.

Tolerances (derived, not fitted): a bf16 rounding is off by at most u = 2^-8 of the value, its
root mean square by u / sqrt(3) = 2.3e-3 of it.  An output passes at most five of them that are
independent: the absorbed query (through scores of standard deviation about 1), the
probabilities, a dequantised latent, the merged latent and the output itself, so its relative
L2 error stays below sqrt(5) * 2.3e-3 = 5.1e-3; 1e-2 leaves a factor of two for scores with a
larger spread.  Element by element an output of size up to 4 is off by at most a few u * 1:
3e-2, the bound of the other parity tests.  float32: 2^-24 in place of 2^-8 in sums of at most
a few hundred terms, below 1e-5.  A token too many or too few changes an output over at most a
few hundred visible tokens by more than its share of the weight, 1 / 300, of an element of
standard deviation 1 / sqrt(300) ... 1: the small windows below make that several times the
bound.
"""

import numpy as np
import pytest
import torch

from tests.helpers import assert_close
from tests.window_helpers import BLOCK, Layer, hidden_tokens, make_cache, store

pytestmark = pytest.mark.gpu

LAYERS = {
    "tiny_f32": dict(dtype="f32", H=4, n_kv=4, d_h=32, r=2, d_c=32),
    "gqa_f32_r3": dict(dtype="f32", H=6, n_kv=2, d_h=24, r=3, d_c=20),
    "smollm": dict(H=9, n_kv=3, d_h=64, d_c=32),
    "smollm_r128": dict(H=9, n_kv=3, d_h=64, d_c=32, cache="int4_r128"),
    "llama_dc256": dict(d_c=256),
    "llama_dc64": dict(d_c=64),
    "llama_dc96": dict(d_c=96),
    "llama_int4": dict(d_c=128, cache="int4"),
    "llama_int4_dc256": dict(d_c=256, cache="int4"),
    "llama_int2": dict(d_c=64, cache="int2"),
    "llama_r128": dict(d_c=128, cache="int4_r128"),
    "gqa64_int4": dict(H=64, n_kv=8, d_h=64, d_c=128, cache="int4"),
    "gqa64": dict(H=64, n_kv=32, d_h=64, d_c=128),
    "one_head_r13": dict(H=1, n_kv=1, d_h=64, r=13, d_c=64),
    "nope": dict(H=8, n_kv=8, d_h=32, r=0, d_c=32),
    # key boxes of 8 KV heads: partly filled ones, two and three query heads per KV head
    "h24_gqa2": dict(H=24, n_kv=12, d_h=32, d_c=64),
    "h27_gqa3": dict(H=27, n_kv=9, d_h=48, d_c=32),
    "h20_dh40": dict(H=20, n_kv=20, d_h=40, d_c=160),
    "h16_int4": dict(H=16, n_kv=16, d_h=32, d_c=192, cache="int4"),
    "h32_gqa8_int2": dict(H=32, n_kv=4, d_h=64, d_c=128, cache="int2"),
}
WINDOWS = [(0, 1), (1, 1), (3, 5), (64, 64), (65, 63), (0, 128), (4, 200), (130, 300), (5000, 7), (0, 5000)]
LENS = [1, 700, 0, 64, 65, 200, 513, 2, 331]


def run_decode(mla, layer, cache, lens, q, n_sink, window, plan=None, out=None):
    own = plan is None
    plan = plan or layer.plan(mla)
    out = torch.full_like(q, float("nan"), device="cuda") if out is None else out
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, q.shape[0]), dtype=torch.uint8, device="cuda")
    mla.mla_decode_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), out, ws,
                          n_sink, window)
    assert mla.mla_device_error(plan) == 0
    if own:
        plan.close()
    return out


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("name", list(LAYERS))
def test_decode_window(name, paged):
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=1)
    B, T_cap = len(LENS), 768
    seqs = [layer.sequence(L) for L in LENS]
    q = layer.queries(B)
    plan = layer.plan(mla)
    for n_sink, window in WINDOWS:
        cache = make_cache(mla, layer, B, T_cap, paged, seed=n_sink + window)
        for b, s in enumerate(seqs):
            store(cache, b, s, hidden_tokens(LENS[b], LENS[b] - 1, n_sink, window))
        got = run_decode(mla, layer, cache, LENS, q, n_sink, window, plan).double().cpu().numpy()
        for b, L in enumerate(LENS):
            if L == 0:
                assert not got[b].any()
                continue
            ref = layer.reference(q[b], seqs[b], L - 1, n_sink, window).numpy()
            assert_close(got[b], ref, layer.dtype, f"{name} sinks {n_sink} window {window} length {L}")
    plan.close()


@pytest.mark.parametrize("kernel", [1, 3])
def test_decode_window_kernels(kernel):
    """Both kernels that have a window, over the same cache."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=128, cache="int4", seed=2)
    lens = [1000, 77]
    seqs = [layer.sequence(L) for L in lens]
    q = layer.queries(2)
    cache = make_cache(mla, layer, 2, 1024, True)
    for b, s in enumerate(seqs):
        store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, 10, 150))
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
    got = run_decode(mla, layer, cache, lens, q, 10, 150, plan).double().cpu().numpy()
    for b, L in enumerate(lens):
        assert_close(got[b], layer.reference(q[b], seqs[b], L - 1, 10, 150).numpy(), "bf16", f"kernel {kernel} {L}")
    plan.close()


@pytest.mark.parametrize("splits", [1, 7, 1000])
def test_decode_window_splits(splits):
    """Any number of workers over the visible tokens, the softmax scale of the config too."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=3, scale=0.05)
    lens = [3000, 1, 700]
    seqs = [layer.sequence(L) for L in lens]
    q = layer.queries(3)
    cache = make_cache(mla, layer, 3, 3008, False)
    for b, s in enumerate(seqs):
        store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, 70, 900))
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_SPLITS, splits)
    got = run_decode(mla, layer, cache, lens, q, 70, 900, plan).double().cpu().numpy()
    for b, L in enumerate(lens):
        assert_close(got[b], layer.reference(q[b], seqs[b], L - 1, 70, 900).numpy(), "bf16", f"splits {splits} {L}")
    plan.close()


def test_full_window_is_decode():
    """A window over everything is mla_decode's attention."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=128, seed=4)
    lens = [900, 130, 1]
    cache = make_cache(mla, layer, 3, 1024, True)
    for b, L in enumerate(lens):
        store(cache, b, layer.sequence(L))
    q = layer.queries(3)
    plan = layer.plan(mla)
    got = run_decode(mla, layer, cache, lens, q, 0, 2 ** 31 - 1, plan)
    sinks = run_decode(mla, layer, cache, lens, q, 2 ** 31 - 1, 1, plan)
    ref = torch.empty_like(got)
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, 3), dtype=torch.uint8, device="cuda")
    mla.mla_decode(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), ref, ws)
    torch.cuda.synchronize()
    for x in (got, sinks):
        assert_close(x.double().cpu().numpy(), ref.double().cpu().numpy(), "bf16")
    plan.close()


CHUNK_LAYERS = ["smollm", "llama_dc256", "llama_dc64", "llama_dc96", "llama_int4", "llama_int4_dc256", "llama_int2", "gqa64",
                "h24_gqa2", "h27_gqa3", "h20_dh40", "h32_gqa8_int2"]


@pytest.mark.parametrize("Q", [1, 2, 5, 70])
@pytest.mark.parametrize("name", CHUNK_LAYERS)
def test_chunk_window(name, Q):
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=5)
    lens = [700, 70, 200, 331]
    B, T_cap = len(lens), 768
    seqs = [layer.sequence(L) for L in lens]
    q = layer.queries(B, Q)
    plan = layer.plan(mla)
    for k, (n_sink, window) in enumerate([(0, 1), (3, 5), (64, 64), (65, 130), (4, 300), (1000, 1), (0, 1000)]):
        cache = make_cache(mla, layer, B, T_cap, k % 2 == 0, seed=k)
        for b, s in enumerate(seqs):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - Q, n_sink, window))
        out = torch.full_like(q, float("nan"), device="cuda")
        ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
        mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(),
                                    out, ws, n_sink, window)
        assert mla.mla_device_error(plan) == 0
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        for b, L in enumerate(lens):
            for i in sorted({0, Q // 2, Q - 1}):
                ref = layer.reference(q[b, i], seqs[b], L - Q + i, n_sink, window).numpy()
                assert_close(got[b, i], ref, "bf16", f"{name} Q {Q} query {i} sinks {n_sink} window {window} length {L}")
    plan.close()


def _exact_layer(cache="same", d_c=32, H=9, n_kv=3, dtype="bf16"):
    """A layer in which scores are exact: W_uk passes the first d_c NoPE dims of the query to the
    latent dims, the softmax scale makes a unit of q . c one unit of log2, the RoPE keys are 0."""
    layer = Layer(dtype=dtype, cache=cache, H=H, n_kv=n_kv, d_h=64, r=4, d_c=d_c, seed=12, scale=float(np.log(2.0)))
    layer.W_uk = torch.zeros_like(layer.W_uk)
    for c in range(d_c):
        layer.W_uk[:, c, c] = 1.0
    layer.W_uv = torch.zeros_like(layer.W_uv)
    for c in range(d_c):
        layer.W_uv[:, c, c] = 1.0
    return layer


def _exact_sequence(layer, L, ramp):
    """Latent 0 of token t is ramp[t] (the score), the others small whole numbers."""
    s = layer.sequence(L)
    g = torch.Generator().manual_seed(5)
    s["c_kv"] = torch.randint(-4, 5, (L, layer.d_c), generator=g).to(layer.td)
    s["c_kv"][:, 0] = torch.as_tensor(ramp).to(layer.td)
    s["c"] = s["c_kv"].double()
    s["kr"] = torch.zeros_like(s["kr"])
    return s


RAMPS = {
    "rising": lambda L: np.minimum(np.arange(L), 200),                    # the maximum moves on and on
    "falling": lambda L: -np.minimum(np.arange(L), 200),
    "jumps": lambda L: np.where(np.arange(L) % 97 == 50, 96, -128) + np.where(np.arange(L) == L - 3, 120, 0),
    "first_low": lambda L: np.where(np.arange(L) % 64 == 0, -240, 16),    # far below the rest of its tile
    "flat": lambda L: np.zeros(L),
}


@pytest.mark.parametrize("ramp", list(RAMPS))
@pytest.mark.parametrize("kind", ["smollm", "llama", "f32"])
def test_score_ranges(kind, ramp):
    """Scores that are whole numbers of log2 units over ranges of up to 368: probabilities are
    powers of two, sums and products exact in float32, so what is left is the output's rounding
    (2^-8 of the value, float32: some 2^-20 of the sums) and, where a probability is below 2^-126
    of the largest, nothing.  Decode over every window kernel, and a chunk."""
    import mha_mla_latent_b200 as mla
    layer = _exact_layer(**{"smollm": dict(), "llama": dict(d_c=32, H=32, n_kv=32), "f32": dict(dtype="f32", H=4, n_kv=4)}[kind])
    lens = [700, 1, 130, 513]
    B, T_cap = len(lens), 768
    seqs = [_exact_sequence(layer, L, RAMPS[ramp](L)) for L in lens]
    q = torch.zeros(B, layer.H, layer.d_h)
    # dims 2k and 2k + 1 of the kept pairs do not reach the latent: score dim 0 must be a NoPE dim
    for h in range(layer.H):
        g = h // (layer.H // layer.n_kv)
        rope = set(np.stack([2 * layer.pairs[g], 2 * layer.pairs[g] + 1], -1).reshape(-1).tolist())
        nope = [i for i in range(layer.d_h) if i not in rope]
        q[:, h, nope[0]] = 1.0
    q = q.to(layer.td)
    eps = 2.0 ** -8 if layer.dtype == "bf16" else 2.0 ** -18
    plan = layer.plan(mla)
    cache = make_cache(mla, layer, B, T_cap, True)
    for b, s in enumerate(seqs):
        store(cache, b, s)
    for kernel in (0, 1) if kind == "f32" else (0, 1, 3):
        mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
        for n_sink, window in [(0, 5000), (3, 100), (70, 300)]:
            got = run_decode(mla, layer, cache, lens, q, n_sink, window, plan).double().cpu()
            for b, L in enumerate(lens):
                ref = layer.reference(q[b], seqs[b], L - 1, n_sink, window)
                worst = ((got[b] - ref).abs() / (ref.abs() * eps + eps / 8)).max().item()
                assert worst <= 1.0, f"{kind} {ramp} kernel {kernel} sinks {n_sink} window {window} length {L}: {worst}"
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, 0)
    if layer.dtype == "bf16":
        Q, use = 5, [0, 2, 3]
        qc = torch.stack([q[b].unsqueeze(0).expand(Q, -1, -1) for b in use]).contiguous()
        sub = make_cache(mla, layer, len(use), T_cap, False)
        for k, b in enumerate(use):
            store(sub, k, seqs[b])
        out = torch.empty_like(qc, device="cuda")
        ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, len(use), Q), dtype=torch.uint8, device="cuda")
        mla.mla_decode_chunk_window(plan, sub.struct, torch.tensor([lens[b] for b in use], dtype=torch.int32, device="cuda"),
                                    qc.cuda(), out, ws, 3, 100)
        assert mla.mla_device_error(plan) == 0
        for k, b in enumerate(use):
            for i in range(Q):
                ref = layer.reference(qc[k, i], seqs[b], lens[b] - Q + i, 3, 100)
                worst = ((out[k, i].double().cpu() - ref).abs() / (ref.abs() * eps + eps / 8)).max().item()
                assert worst <= 1.0, f"chunk {kind} {ramp} length {lens[b]} query {i}: {worst}"
    plan.close()


@pytest.mark.parametrize("B,splits", [(100, 1), (700, 0), (300, 2)])
def test_many_short_sequences(B, splits):
    """More pieces per worker than its list holds, more sequences than threads, empty ones among them."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=13)
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 200, size=B).tolist()
    seq = layer.sequence(200)
    cache = make_cache(mla, layer, B, 256, B != 300, seed=1)
    for b, L in enumerate(lens):
        if L:
            store(cache, b, {k: (v[:L] if torch.is_tensor(v) else v) for k, v in seq.items()} | {"L": L})
    q = layer.queries(B)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_SPLITS, splits)
    got = run_decode(mla, layer, cache, lens, q, 20, 150, plan).double().cpu().numpy()
    for b in list(range(0, B, B // 12)) + [B - 1]:
        if lens[b] == 0:
            assert not got[b].any()
        else:
            assert_close(got[b], layer.reference(q[b], seq, lens[b] - 1, 20, 150).numpy(), "bf16", f"{B} {splits} {b}")
    plan.close()


@pytest.mark.parametrize("name", ["llama_dc96", "llama_int4_dc256", "llama_int2", "gqa64"])
def test_chunk_window_head_rows(name):
    """The head-row units (MLA_OPT_DECODE_KERNEL 3), which also serve the head dims that the one-launch form lacks."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=16)
    B, Q = 3, 20
    lens = [20, 131, 390]
    seqs = [layer.sequence(L) for L in lens]
    cache = make_cache(mla, layer, B, 512, True)
    for b, s in enumerate(seqs):
        store(cache, b, s)
    q = layer.queries(B, Q)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, 3)
    out = torch.full_like(q, float("nan"), device="cuda")
    ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
    for n_sink, window in [(0, 1), (5, 120), (70, 200)]:
        mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), out, ws, n_sink, window)
        assert mla.mla_device_error(plan) == 0
        got = out.double().cpu().numpy()
        for b, L in enumerate(lens):
            for i in (0, Q // 2, Q - 1):
                ref = layer.reference(q[b, i], seqs[b], L - Q + i, n_sink, window).numpy()
                assert_close(got[b, i], ref, "bf16", f"{name} sinks {n_sink} window {window} seq {b} query {i}")
    plan.close()


@pytest.mark.parametrize("B,Q,name", [(24, 3, "llama_dc64"), (1, 130, "llama_dc64"), (2, 33, "smollm"), (30, 2, "smollm")])
def test_chunk_window_unit_shapes(B, Q, name):
    """Numbers of sequences and queries that make the chunk's units of one, two and four KV heads."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=14)
    rng = np.random.default_rng(Q)
    lens = rng.integers(Q, 400, size=B).tolist()
    seq = layer.sequence(400)
    cache = make_cache(mla, layer, B, 512, True)
    for b, L in enumerate(lens):
        store(cache, b, {k: (v[:L] if torch.is_tensor(v) else v) for k, v in seq.items()} | {"L": L})
    q = layer.queries(B, Q)
    plan = layer.plan(mla)
    out = torch.full_like(q, float("nan"), device="cuda")
    ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
    mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), out, ws, 5, 120)
    assert mla.mla_device_error(plan) == 0
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    for b in {0, B // 2, B - 1}:
        for i in {0, Q // 2, Q - 1}:
            ref = layer.reference(q[b, i], seq, lens[b] - Q + i, 5, 120).numpy()
            assert_close(got[b, i], ref, "bf16", f"{name} {B} {Q} seq {b} query {i}")
    plan.close()


def test_without_launch_overlap():
    """Plain stream order gives the same bits."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=128, cache="int4", seed=15)
    lens = [600, 333]
    cache = make_cache(mla, layer, 2, 640, True)
    for b, L in enumerate(lens):
        store(cache, b, layer.sequence(L))
    q = layer.queries(2)
    plan = layer.plan(mla)
    a = run_decode(mla, layer, cache, lens, q, 3, 400, plan)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_OVERLAP_LAUNCH, 0)
    b = run_decode(mla, layer, cache, lens, q, 3, 400, plan)
    assert torch.equal(a, b)
    plan.close()


def _poison(cache):
    """Every row as an earlier owner may have left it: not finite."""
    for a in (cache.c_kv, cache.c_scales, cache.k_rope):
        if a is not None:
            a.fill_(float("nan") if a.is_floating_point() else 0x77)


@pytest.mark.parametrize("T_cap", [200, 333])
@pytest.mark.parametrize("name", ["tiny_f32", "smollm", "llama_dc256", "llama_dc64", "llama_int4", "llama_int2"])
def test_stale_rows_and_odd_capacity(name, T_cap):
    """Sequences that end inside a tile, the tile in the next sequence or behind the array; every
    row that is not a visible token holds NaN.  The largest n_sink and window too."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=17)
    lens = [T_cap, 70, T_cap - 5, 9, T_cap]
    B, Q, big = len(lens), 7, 2 ** 31 - 1
    seqs = [layer.sequence(L) for L in lens]
    plan = layer.plan(mla)
    q, qc = layer.queries(B), layer.queries(B, Q)
    for n_sink, window in [(3, 90), (0, 1), (70, 31), (big, big), (0, big)]:
        cache = make_cache(mla, layer, B, T_cap, False)
        _poison(cache)
        for b, s in enumerate(seqs):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, n_sink, window))
        got = run_decode(mla, layer, cache, lens, q, n_sink, window, plan).double().cpu().numpy()
        for b, L in enumerate(lens):
            ref = layer.reference(q[b], seqs[b], L - 1, n_sink, window).numpy()
            assert_close(got[b], ref, layer.dtype, f"{name} {T_cap} sinks {n_sink} window {window} length {L}")
        if layer.dtype != "bf16":
            continue
        for b, s in enumerate(seqs):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - Q, n_sink, window))
        out = torch.empty_like(qc, device="cuda")
        ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
        mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), qc.cuda(),
                                    out, ws, n_sink, window)
        assert mla.mla_device_error(plan) == 0
        for b, L in enumerate(lens):
            for i in (0, Q - 1):
                ref = layer.reference(qc[b, i], seqs[b], L - Q + i, n_sink, window).numpy()
                assert_close(out[b, i].double().cpu().numpy(), ref, "bf16", f"{name} {T_cap} chunk {n_sink} {window} {L} {i}")
    plan.close()


@pytest.mark.parametrize("name", ["smollm", "llama_dc256", "llama_int4", "tiny_f32"])
@pytest.mark.parametrize("splits", [0, 1])
def test_a_bad_sequence_stays_alone(name, splits):
    """A sequence whose visible rows are not finite changes no other sequence's bits, with its
    pieces beside theirs in the same worker too."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=18)
    lens = [300, 500, 129, 700]
    B, T_cap, Q = len(lens), 768, 6
    seqs = [layer.sequence(L) for L in lens]
    q, qc = layer.queries(B), layer.queries(B, Q)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_SPLITS, splits)
    outs = []
    for bad in (False, True):
        cache = make_cache(mla, layer, B, T_cap, True)
        for b, s in enumerate(seqs):
            store(cache, b, s, torch.arange(lens[b]) if bad and b == 1 else None)
        o = [run_decode(mla, layer, cache, lens, q, 5, 1000, plan), run_decode(mla, layer, cache, lens, q, 5, 150, plan)]
        if layer.dtype == "bf16":
            out = torch.empty_like(qc, device="cuda")
            ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), dtype=torch.uint8, device="cuda")
            mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        qc.cuda(), out, ws, 5, 150)
            o.append(out)
        outs.append(o)
    for good, bad in zip(*outs):
        for b in (0, 2, 3):
            assert torch.isfinite(good[b].float()).all() and torch.equal(good[b], bad[b])
        assert not torch.isfinite(bad[1].float()).any()
    plan.close()


def test_short_sequences_in_a_chunk():
    """Sequences shorter than the chunk (empty ones too) are flagged and give zeros; the others are computed."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=19)
    lens, Q = [0, 5, 300, 257, 8], 8
    cache = make_cache(mla, layer, 5, 256, True)
    seq = layer.sequence(256)
    for b in (0, 1, 3, 4):
        store(cache, b, seq)
    lens[2] = 256
    store(cache, 2, seq)
    q = layer.queries(5, Q)
    plan = layer.plan(mla)
    for kernel in (0, 3):
        mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
        out = torch.full_like(q, float("nan"), device="cuda")
        ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, 5, Q), dtype=torch.uint8, device="cuda")
        mla.mla_decode_chunk_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(),
                                    out, ws, 4, 40)
        assert mla.mla_device_error(plan) == mla.MLA_DEVERR_SEQ_LEN
        got = out.double().cpu().numpy()
        assert not got[0].any() and not got[1].any() and not got[3].any()
        for b in (2, 4):
            for i in (0, Q - 1):
                ref = layer.reference(q[b, i], seq, lens[b] - Q + i, 4, 40).numpy()
                assert_close(got[b, i], ref, "bf16", f"kernel {kernel} {b} {i}")
    plan.close()


def test_out_of_range_length():
    """A length beyond the capacity is flagged and treated as empty; the others are computed."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=6)
    cache = make_cache(mla, layer, 3, 256, False)
    seq = layer.sequence(100)
    for b in range(3):
        store(cache, b, seq)
    q = layer.queries(3)
    plan = layer.plan(mla)
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, 3), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"), device="cuda")
    mla.mla_decode_window(plan, cache.struct, torch.tensor([257, 100, -1], dtype=torch.int32, device="cuda"), q.cuda(),
                          out, ws, 4, 40)
    assert mla.mla_device_error(plan) == mla.MLA_DEVERR_SEQ_LEN
    got = out.double().cpu().numpy()
    assert not got[0].any() and not got[2].any()
    assert_close(got[1], layer.reference(q[1], seq, 99, 4, 40).numpy(), "bf16")
    plan.close()


def test_long_cache_offsets():
    """Rows behind 2^32 bytes of every array of a paged cache, at positions near 2^20."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import LatentCache
    layer = Layer(d_c=256, seed=7)
    n_blocks, L, window = 70000, (1 << 20) - 30, 300
    C = (1 << 20) // BLOCK
    table = np.full((1, C), -1, dtype=np.int32)
    table[0, -4:] = [69999, 66001, 69998, 3]
    table[0, 0] = 69990
    cache = LatentCache(layer.config(mla), 1, 1 << 20, "cuda", block_table=table, n_blocks=n_blocks)
    assert cache.c_kv.numel() * 2 > 2 ** 32 and cache.k_rope.numel() * 2 > 2 ** 32
    seq = layer.sequence(2 + window)          # the two sinks, then the window
    tail = {k: v[2:] for k, v in seq.items() if k != "L"}
    cache.set_latent_rows(0, 0, seq["c_kv"][:2])
    cache.set_k_rope_tokens(0, 0, seq["kr"][:2])
    cache.set_latent_rows(0, L - window, tail["c_kv"])
    cache.set_k_rope_tokens(0, L - window, tail["kr"])
    q = layer.queries(1)
    got = run_decode(mla, layer, cache, [L], q, 2, window).double().cpu().numpy()
    # the same tokens as a short sequence whose query is rotated at the far position
    s = dict(c=seq["c"], kr=seq["kr"])
    far = _reference_at(layer, q[0], s, L - 1)
    assert_close(got[0], far.numpy(), "bf16")


def _reference_at(layer, q, seq, p):
    """Every row of `seq` visible, the query rotated at p."""
    q = q.double().clone()
    turned = q.clone()
    for h in range(layer.H):
        k = layer.pairs[h // (layer.H // layer.n_kv)]
        ang = torch.from_numpy(p * 10000.0 ** (-2.0 * k / layer.d_h))
        n = seq["c"].shape[0]
        back = torch.from_numpy((n - 1) * 10000.0 ** (-2.0 * k / layer.d_h))   # what reference() turns by
        d = ang - back
        x, y = q[h, 2 * k], q[h, 2 * k + 1]
        turned[h, 2 * k], turned[h, 2 * k + 1] = x * d.cos() - y * d.sin(), x * d.sin() + y * d.cos()
    return layer.reference(turned, seq, seq["c"].shape[0] - 1, 0, seq["c"].shape[0])


def test_graph_replay_and_two_streams():
    """A captured call replayed over changed lengths, and two plans' calls at once on two streams."""
    import mha_mla_latent_b200 as mla
    layers = [Layer(d_c=64, seed=8), Layer(d_c=128, cache="int4", seed=9)]
    L = 600
    seqs = [layer.sequence(L) for layer in layers]
    caches = [make_cache(mla, layer, 1, 640, True) for layer in layers]
    for c, s in zip(caches, seqs):
        store(c, 0, s)
    plans = [layer.plan(mla) for layer in layers]
    qs = [layer.queries(1).cuda() for layer in layers]
    outs = [torch.empty_like(q) for q in qs]
    wss = [torch.empty(mla.mla_decode_workspace_bytes(p, 1), dtype=torch.uint8, device="cuda") for p in plans]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    call = lambda k: mla.mla_decode_window(plans[k], caches[k].struct, lens, qs[k], outs[k], wss[k], 3, 100)  # noqa: E731
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                call(k)
    torch.cuda.synchronize()
    for k in (0, 1):
        ref = layers[k].reference(qs[k][0].cpu(), seqs[k], L - 1, 3, 100).numpy()
        assert_close(outs[k][0].double().cpu().numpy(), ref, "bf16", f"stream {k}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for n in (600, 37, 471):
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref = layers[0].reference(qs[0][0].cpu(), seqs[0], n - 1, 3, 100).numpy()
        assert_close(outs[0][0].double().cpu().numpy(), ref, "bf16", f"replay {n}")
    for p in plans:
        assert mla.mla_device_error(p) == 0
        p.close()


@pytest.mark.parametrize("name,skip,chunk", [("llama_dc256", 1, False), ("llama_dc256", 2, False), ("llama_int4", 1, False),
                                             ("llama_dc64", 2, True), ("llama_int4_dc256", 1, True)])
def test_wait_runs_out_then_plan_recovers(name, skip, chunk):
    """A copy that never comes: every wait behind it is bounded, the call comes back and reports
    it, and the next one on the same plan is right."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=20)
    lens, Q = [512, 300], 3 if chunk else 1
    seqs = [layer.sequence(L) for L in lens]
    cache = make_cache(mla, layer, 2, 512, True)
    for b, s in enumerate(seqs):
        store(cache, b, s)
    q = layer.queries(2, Q)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_SPLITS, 1)   # (decode) one CTA with every tile
    out = torch.empty_like(q, device="cuda")
    ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, 2, Q), dtype=torch.uint8, device="cuda")
    call = lambda: mla.mla_decode_chunk_window(  # noqa: E731
        plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), out, ws, 10, 400)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_WAIT_LIMIT_US, 2000)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_TEST_SKIP_COPY, skip)
    call()
    assert mla.mla_device_error(plan) & mla.MLA_DEVERR_TIMEOUT
    mla.mla_plan_set_option(plan, mla.MLA_OPT_TEST_SKIP_COPY, 0)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_WAIT_LIMIT_US, 1_000_000)
    out.fill_(float("nan"))
    call()
    assert mla.mla_device_error(plan) == 0
    for b, L in enumerate(lens):
        for i in range(Q):
            ref = layer.reference(q[b, i], seqs[b], L - Q + i, 10, 400).numpy()
            assert_close(out[b, i].double().cpu().numpy(), ref, "bf16", f"{name} after the timeout {b} {i}")
    plan.close()


def test_refusals():
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=10)
    plan = layer.plan(mla)
    cache = make_cache(mla, layer, 2, 256, False)
    lens = torch.full((2,), 100, dtype=torch.int32, device="cuda")
    q = layer.queries(2).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, 2), dtype=torch.uint8, device="cuda")
    call = lambda S, W, w=ws: mla.mla_decode_window(plan, cache.struct, lens, q, out, w, S, W, check=False)  # noqa: E731
    assert call(0, 0) == mla.MLA_ERR_INVALID_ARG and call(-1, 4) == mla.MLA_ERR_INVALID_ARG
    assert call(0, -5) == mla.MLA_ERR_INVALID_ARG
    assert call(0, 4, ws[:256]) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    qc = q.unsqueeze(1).expand(2, 300, 32, 128).contiguous()
    oc = torch.empty_like(qc)
    chunk = lambda q_, W: mla.mla_decode_chunk_window(plan, cache.struct, lens, q_, oc, ws, 0, W, check=False)  # noqa: E731
    assert chunk(qc, 4) == mla.MLA_ERR_INVALID_ARG                       # Q > T_cap
    assert chunk(qc[:, :8].contiguous(), 0) == mla.MLA_ERR_INVALID_ARG
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, 2)
    assert call(0, 4) == mla.MLA_ERR_UNSUPPORTED
    assert chunk(qc[:, :8].contiguous(), 4) == mla.MLA_ERR_UNSUPPORTED
    plan.close()
    with pytest.raises(mla.MlaError):
        ring = Layer(d_c=128, cache="int4_r128", seed=11)
        rp = ring.plan(mla)
        rc = make_cache(mla, ring, 2, 256, False)
        mla.mla_decode_chunk_window(rp, rc.struct, lens, qc[:, :8].contiguous(), oc, ws, 0, 4)


def test_tensors_that_do_not_fit_are_refused():
    """Shapes, types and places that the kernels could not read safely: refused on the host."""
    import mha_mla_latent_b200 as mla
    layer = Layer(d_c=64, seed=23)
    plan = layer.plan(mla)
    cache = make_cache(mla, layer, 2, 256, False)
    lens = torch.full((2,), 100, dtype=torch.int32, device="cuda")
    q = layer.queries(2).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(mla.mla_decode_chunk_workspace_bytes(plan, 2, 3), dtype=torch.uint8, device="cuda")
    assert mla.mla_decode_window(plan, cache.struct, lens, q, out, ws, 0, 4) == mla.MLA_OK
    args = dict(p=plan, c=cache.struct, l=lens, q=q, o=out, w=ws, s=0, n=4)
    run = lambda f, **kw: f(*[{**args, **kw}[k] for k in "pclqowsn"])  # noqa: E731
    host = mla.cache_struct(torch.zeros(2, 256, 64, dtype=torch.bfloat16), None, cache.k_rope, 2, 256)
    for kw in (dict(l=lens[:1]), dict(l=lens.long()), dict(l=lens.cpu()), dict(q=q.cpu()), dict(q=q.float()), dict(o=out[:1]),
               dict(o=out.cpu()), dict(o=out.float()), dict(w=ws.cpu()), dict(c=host), dict(q=q[:, :16]), dict(q=q[None]),
               dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(w=ws[::2])):
        with pytest.raises(ValueError):
            run(mla.mla_decode_window, **kw)
    with pytest.raises(ValueError):
        run(mla.mla_decode_chunk_window)          # [B][H][d_h] where the chunk's [B][Q][H][d_h] belongs
    torch.cuda.synchronize()
    assert mla.mla_device_error(plan) == 0
    plan.close()


@pytest.mark.parametrize("B", [2, 64])
def test_default_kernel_keeps_up_with_a_forced_one(B):
    """Layers with more heads than the windowed tensor-core kernel takes: the one-launch form is for
    few rows only (at 64 sequences it takes seven times the head-row kernel's time)."""
    import mha_mla_latent_b200 as mla
    layer = Layer(H=64, n_kv=32, d_h=64, d_c=128, seed=24)
    cache = make_cache(mla, layer, B, 1100, False)
    cache.c_kv.normal_()
    cache.k_rope.normal_()
    plan = layer.plan(mla)
    q = layer.queries(B).cuda()
    out = torch.empty_like(q)
    lens = torch.full((B,), 1100, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, B), dtype=torch.uint8, device="cuda")
    best = {}
    for kernel in (0, 3):
        mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
        graph = torch.cuda.CUDAGraph()
        mla.mla_decode_window(plan, cache.struct, lens, q, out, ws, 0, 1100)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(10):
                mla.mla_decode_window(plan, cache.struct, lens, q, out, ws, 0, 1100)
        times = []
        for _ in range(6):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            graph.replay()
            t[1].record()
            torch.cuda.synchronize()
            times.append(t[0].elapsed_time(t[1]))
        best[kernel] = min(times[1:])
    assert best[0] <= 1.5 * best[3], best
    plan.close()
