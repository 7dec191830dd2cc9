"""The framework's own append, step, decode and chunk through tables that a BlockPool makes.

Two layers share one pool; prompts are forked, samples grow with copy on write, blocks behind the
window are released and the pool is compacted on the way.  A second pair of caches, contiguous and
never shared or trimmed, gets the same tokens: what the pool's cache gives is the same, bit for bit
(the kernels and their splits depend on the lengths only).
"""

import numpy as np
import pytest
import torch

from tests.helpers import assert_close
from tests.test_gpu_window import LAYERS, run_decode
from tests.window_helpers import Layer, hidden_tokens, make_cache, store

pytestmark = pytest.mark.gpu

HIDDEN = 64


def full_plan(mla, layer, seed):
    """A plan with random down-projections, so that the append stores real rows."""
    g = torch.Generator().manual_seed(seed)
    W = [(torch.randn(HIDDEN, n, generator=g) * HIDDEN ** -0.5).to(layer.td) for n in (layer.d_c, layer.n_kv * layer.d_h)]
    return mla.mla_plan_create(layer.config(mla), *W, torch.from_numpy(layer.pairs), layer.W_uk, layer.W_uv)


@pytest.mark.parametrize("kinds", [(dict(d_c=64), dict(d_c=128, cache="int4")), (dict(d_c=128, cache="int4_r128"), dict(d_c=96)),
                                   (dict(H=9, n_kv=3, d_h=64, d_c=64, cache="int2"), dict(H=9, n_kv=3, d_h=64, d_c=32))], ids=str)
def test_serving_with_the_frameworks_append(kinds):
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool, LatentCache
    layers = [Layer(**k, seed=30 + i) for i, k in enumerate(kinds)]
    plans = [full_plan(mla, layer, i) for i, layer in enumerate(layers)]
    B, T_cap, n_sink, window = 6, 1024, 3, 150
    prompts = [200, 333]
    pool = BlockPool(B, T_cap, 60)
    pooled = [pool.layer(layer.config(mla)) for layer in layers]
    flat = [LatentCache(layer.config(mla), B, T_cap, "cuda") for layer in layers]
    g = torch.Generator().manual_seed(5)
    i32 = lambda v: torch.as_tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    rows = lambda n: torch.randn(n, HIDDEN, generator=g).to(torch.bfloat16).cuda()  # noqa: E731

    def append(caches, x, seq, pos):
        for plan, c in zip(plans, caches):
            mla.mla_append(plan, x, i32(seq), i32(pos), c.struct)

    def ws(plan, Q):
        n = max(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), mla.mla_decode_workspace_bytes(plan, B))
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def both(call, what):
        """`call(plan, cache, layer)` for every layer, on the pool's cache and on the contiguous one."""
        for plan, a, b, layer in zip(plans, pooled, flat, layers):
            state = g.get_state()
            x = call(plan, a, layer)
            g.set_state(state)
            y = call(plan, b, layer)
            assert torch.isfinite(x.float()).all() and torch.equal(x, y), what

    # prompts, appended once into the pool and for every sample into the contiguous caches
    pool.reserve([0] * B, prompts + [0] * 4)
    for b, P in enumerate(prompts):
        x = rows(P)
        append(pooled, x, [b] * P, range(P))
        for s in range(b, B, 2):
            append(flat, x, [s] * P, range(P))
    pool.fork([0, 0, 1, 1], [2, 4, 3, 5], prompts + [0] * 4)
    lens = np.array([prompts[b % 2] for b in range(B)])
    assert pool.in_use() == 2 + 3

    for step in range(40):
        Q = 1 if step % 5 else 7
        pool.reserve(lens, lens + Q)
        lens = lens + Q
        seq = [b for b in range(B) for _ in range(Q)]
        pos = [int(lens[b]) - Q + i for b in range(B) for i in range(Q)]
        x = rows(B * Q)
        if Q == 1 and step < 4:    # the whole prefix is still there: append and decode in one call
            both(lambda plan, c, layer: _step(mla, plan, c, lens, x, layer, g, ws(plan, 1), i32), f"step {step}")
        else:
            append(pooled, x, seq, pos)
            append(flat, x, seq, pos)
        if step % 7 == 4:
            pool.trim(lens, n_sink, window + 7)   # the next chunk's first query sees `window` tokens too
        if step % 11 == 5:
            pool.compact()
            assert int(torch.nonzero(pool.refs).max()) == pool.in_use() - 1
        both(lambda plan, c, layer: _window(mla, plan, c, lens, layer, g, ws(plan, 1), i32, n_sink, window), f"window {step}")
        if Q > 1:
            for plan, a, b, layer in zip(plans, pooled, flat, layers):
                if layer.cache == "int4_r128":
                    continue   # (no chunks over the residual window)
                q = torch.randn(B, Q, layer.H, layer.d_h, generator=g).to(torch.bfloat16).cuda()
                o = [torch.empty_like(q) for _ in range(2)]
                for c, out in zip((a, b), o):
                    mla.mla_decode_chunk_window(plan, c.struct, i32(lens), q, out, ws(plan, Q), n_sink, window)
                assert torch.isfinite(o[0].float()).all() and torch.equal(*o), f"chunk {step}"
        assert pool.errors() == 0 and all(mla.mla_device_error(p) == 0 for p in plans), step
    named = pool.table[pool.table >= 0].long()
    assert torch.equal(torch.bincount(named.cpu(), minlength=60).int(), pool.refs.cpu())
    assert (pool.table == -1).any()
    pool.trim([0] * B, 0, 0)
    assert pool.in_use() == 0
    for p in plans:
        p.close()


def _step(mla, plan, c, lens, x, layer, g, ws, i32):
    q = torch.randn(len(lens), layer.H, layer.d_h, generator=g).to(torch.bfloat16).cuda()
    out = torch.empty_like(q)
    mla.mla_decode_step(plan, c.struct, i32(lens), x, q, out, ws)
    return out


def _window(mla, plan, c, lens, layer, g, ws, i32, n_sink, window):
    q = torch.randn(len(lens), layer.H, layer.d_h, generator=g).to(torch.bfloat16).cuda()
    out = torch.empty_like(q)
    mla.mla_decode_window(plan, c.struct, i32(lens), q, out, ws, n_sink, window)
    return out


def test_a_full_pool_leaves_the_table_and_the_rows():
    """A reserve that the pool cannot serve changes nothing but the status; appends that are held back
    on it, without the host, leave every row as it was."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=64, seed=33)
    plan = full_plan(mla, layer, 3)
    pool = BlockPool(2, 512, 3)
    cache = pool.layer(layer.config(mla))
    g = torch.Generator().manual_seed(7)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool.reserve([0, 0], [300, 0])
    mla.mla_append(plan, torch.randn(300, HIDDEN, generator=g).to(torch.bfloat16).cuda(), i32([0] * 300), i32(range(300)), cache.struct)
    pool.fork([0], [1], [300, 0])
    before = cache.c_kv.clone(), pool.table.clone(), pool.refs.clone()
    pool.reserve([300, 300], [301, 301])     # a copy of the shared block, and no block is free
    full = (pool.status[1] & mla.MLA_DEVERR_POOL) != 0
    x = torch.randn(2, HIDDEN, generator=g).to(torch.bfloat16).cuda()
    mla.mla_append(plan, x, i32([0, 1]), torch.where(full, -1, i32([300, 300])).int(), cache.struct)
    torch.cuda.synchronize()
    for a, b in zip(before, (cache.c_kv, pool.table, pool.refs)):
        assert torch.equal(a, b)
    assert pool.errors() == mla.MLA_DEVERR_POOL and mla.mla_device_error(plan) == mla.MLA_DEVERR_APPEND_SLOT
    plan.close()


@pytest.mark.parametrize("name", ["llama_int4_dc256", "gqa64_int4_dc256"])
def test_decode_and_chunk_of_the_widest_4_bit_latents(name):
    """Shapes whose rings only fit when they are shallow (one key stage, two code stages), without a
    window: mla_decode_chunk, and mla_decode with 64 heads."""
    import mha_mla_latent_b200 as mla
    kw = LAYERS.get(name) or dict(H=64, n_kv=32, d_h=64, d_c=256, cache="int4")
    layer = Layer(**kw, seed=34)
    lens, Q = [700, 70, 331], 13
    B, T_cap, big = len(lens), 768, 100000
    seqs = [layer.sequence(L) for L in lens]
    plan = layer.plan(mla)
    for paged in (False, True):
        cache = make_cache(mla, layer, B, T_cap, paged)
        for b, s in enumerate(seqs):
            store(cache, b, s)
        L32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q, qc = layer.queries(B), layer.queries(B, Q)
        out, oc = torch.empty_like(q, device="cuda"), torch.empty_like(qc, device="cuda")
        ws = torch.empty(max(mla.mla_decode_chunk_workspace_bytes(plan, B, Q), mla.mla_decode_workspace_bytes(plan, B)),
                         dtype=torch.uint8, device="cuda")
        mla.mla_decode(plan, cache.struct, L32, q.cuda(), out, ws)
        mla.mla_decode_chunk(plan, cache.struct, L32, qc.cuda(), oc, ws)
        assert mla.mla_device_error(plan) == 0
        for b, L in enumerate(lens):
            assert_close(out[b].double().cpu().numpy(), layer.reference(q[b], seqs[b], L - 1, 0, big).numpy(), "bf16", f"{name} {L}")
            for i in (0, 6, Q - 1):
                ref = layer.reference(qc[b, i], seqs[b], L - Q + i, 0, big).numpy()
                assert_close(oc[b, i].double().cpu().numpy(), ref, "bf16", f"{name} {L} query {i}")
    plan.close()


@pytest.mark.parametrize("name,kernel", [("gqa64", 0), ("gqa64", 3), ("tiny_f32", 0), ("nope", 0), ("one_head_r13", 0),
                                         ("gqa_f32_r3", 0), ("smollm_r128", 0), ("gqa64_int4", 1)])
def test_long_windows_on_the_other_kernels(name, kernel):
    """More visible tokens than the one-launch form takes, on the layers without the windowed
    tensor-core kernel; hidden rows hold NaN."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**LAYERS[name], seed=35)
    lens = [2000, 1400, 1153, 40]
    B, T_cap = len(lens), 2048
    seqs = [layer.sequence(L) for L in lens]
    q = layer.queries(B)
    plan = layer.plan(mla)
    mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
    for n_sink, window in [(70, 1200), (0, 1153), (33, 1601)]:
        cache = make_cache(mla, layer, B, T_cap, True)
        for b, s in enumerate(seqs):
            store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, n_sink, window))
        got = run_decode(mla, layer, cache, lens, q, n_sink, window, plan).double().cpu().numpy()
        for b, L in enumerate(lens):
            ref = layer.reference(q[b], seqs[b], L - 1, n_sink, window).numpy()
            assert_close(got[b], ref, layer.dtype, f"{name} {kernel} sinks {n_sink} window {window} length {L}")
    plan.close()


@pytest.mark.parametrize("kind", [dict(d_c=64), dict(d_c=128, cache="int4"), dict(d_c=128, cache="int4_r128"), dict(d_c=64, cache="int2"),
                                  dict(dtype="f32", H=4, n_kv=4, d_h=32, r=2, d_c=32)], ids=str)
def test_append_without_a_block_touches_no_other_sequence(kind):
    """A token whose column has no block (no reserve, or trimmed since) goes nowhere: block 0 belongs to
    whoever holds it."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(**kind, seed=36)
    plan = full_plan(mla, layer, 6)
    pool = BlockPool(2, 1024, 8)
    cache = pool.layer(layer.config(mla))
    g = torch.Generator().manual_seed(8)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = lambda n: torch.randn(n, HIDDEN, generator=g).to(layer.td).cuda()  # noqa: E731
    pool.reserve([0, 0], [300, 0])
    assert pool.table[0, :3].tolist() == [0, 1, 2]
    mla.mla_append(plan, rows(300), i32([0] * 300), i32(range(300)), cache.struct)
    arrays = [a for a in (cache.c_kv, cache.c_scales, cache.k_rope) if a is not None]
    before = [a.clone() for a in arrays]
    for n in (1, 40, 500):       # each form of the append
        mla.mla_append(plan, rows(n), i32([1] * n), i32(range(n)), cache.struct)
        assert mla.mla_device_error(plan) == mla.MLA_DEVERR_BLOCK
        assert all(torch.equal(a, b) for a, b in zip(arrays, before)), n
    q = torch.randn(2, layer.H, layer.d_h, generator=g).to(layer.td).cuda()
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, 2), dtype=torch.uint8, device="cuda")
    mla.mla_decode_step(plan, cache.struct, i32([300, 5]), rows(2), q, torch.empty_like(q), ws)   # row 0 rewrites token 299
    assert mla.mla_device_error(plan) == mla.MLA_DEVERR_BLOCK
    for a, b in zip(arrays, before):
        b[2, 299 % 128] = a[2, 299 % 128]
        assert torch.equal(a, b)
    plan.close()


@pytest.mark.parametrize("n", [1, 40, 128])
def test_append_without_a_block_leaves_the_ring(n):
    """The token takes no slot of its sequence's residual window either: the slot still holds one of the
    newest tokens."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=128, cache="int4_r128", seed=37)
    plan = full_plan(mla, layer, 7)
    pool = BlockPool(2, 1024, 8)
    cache = pool.layer(layer.config(mla))
    g = torch.Generator().manual_seed(9)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = lambda k: torch.randn(k, HIDDEN, generator=g).to(layer.td).cuda()  # noqa: E731
    pool.reserve([0, 0], [256, 130])
    mla.mla_append(plan, rows(386), i32([0] * 256 + [1] * 130), i32([*range(256), *range(130)]), cache.struct)
    assert mla.mla_device_error(plan) == 0
    assert cache.resid_pos[0].tolist() == list(range(128, 256))
    ring, pos = cache.c_resid.clone(), cache.resid_pos.clone()
    mla.mla_append(plan, rows(n), i32([0] * n), i32(range(256, 256 + n)), cache.struct)   # no block from 256 on
    assert mla.mla_device_error(plan) == mla.MLA_DEVERR_BLOCK
    assert torch.equal(cache.resid_pos, pos) and torch.equal(cache.c_resid, ring)
    q = torch.randn(2, layer.H, layer.d_h, generator=g).to(layer.td).cuda()
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, 2), dtype=torch.uint8, device="cuda")
    mla.mla_decode_step(plan, cache.struct, i32([257, 131]), rows(2), q, torch.empty_like(q), ws)
    assert mla.mla_device_error(plan) == mla.MLA_DEVERR_BLOCK
    assert torch.equal(cache.resid_pos[0], pos[0]) and torch.equal(cache.c_resid[0], ring[0])
    assert cache.resid_pos[1, 2].item() == 130   # the other sequence's token has a block
    plan.close()
