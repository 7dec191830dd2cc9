"""Refusals of the window and block entry points that need no GPU: bad arguments come back with
the documented status before anything touches the device."""

import ctypes

import pytest
import torch

P = 1 << 20   # a well-aligned address that is never read


@pytest.fixture(scope="module")
def mla():
    from mha_mla_latent_b200 import build
    build.build()
    import mha_mla_latent_b200._lib as lib
    return lib


def test_window_calls_need_a_plan(mla):
    cache = mla.MlaCache(4096, None, 8192, 2, 128)
    c = ctypes.byref(cache)
    assert mla._lib.mla_decode_window(None, c, P, P, 1, 0, 4, P, P, 1 << 20, None) == mla.MLA_ERR_INVALID_ARG
    assert mla._lib.mla_decode_chunk_window(None, c, P, P, 1, 2, 0, 4, P, P, 1 << 20, None) == mla.MLA_ERR_INVALID_ARG


def test_workspace_of_invalid_sizes(mla):
    f = mla.mla_blocks_workspace_bytes
    assert f(0, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == f(1, 1, (1 << 24) + 1) == f(1 << 20, 1 << 11, 1) == 0
    assert f(1, 1, 1) > 0 and f(3, 5, 100) >= 4 * (2 * 3 + 2 * 100)


def blocks(mla, name, **kw):
    """One call with well-formed fake pointers, `kw` replacing some of them."""
    a = dict(table=P, refs=2 * P, B=4, n_cols=8, n_blocks=100, src=3 * P, dst=4 * P, n=2, seq_lens=5 * P, new_lens=6 * P,
             table_out=7 * P, refs_out=8 * P, copies=9 * P, max_copies=50, status=10 * P, ws=11 * P, ws_bytes=1 << 20,
             n_sink=0, window=4)
    a.update(kw)
    order = {"fork": "table refs B n_cols n_blocks src dst n seq_lens table_out refs_out status",
             "reserve": "table refs B n_cols n_blocks seq_lens new_lens table_out refs_out copies max_copies status ws ws_bytes",
             "trim": "table refs B n_cols n_blocks seq_lens n_sink window table_out refs_out status",
             "compact": "table refs B n_cols n_blocks table_out refs_out copies max_copies status ws ws_bytes"}[name]
    return getattr(mla._lib, "mla_blocks_" + name)(*[a[k] for k in order.split()], None)


@pytest.mark.parametrize("name", ["fork", "reserve", "trim", "compact"])
def test_block_calls_refuse_bad_arguments(mla, name):
    bad = [dict(table=None), dict(refs=None), dict(table_out=None), dict(refs_out=None), dict(status=None), dict(B=0),
           dict(n_cols=-1), dict(n_blocks=0), dict(n_blocks=(1 << 24) + 1), dict(table_out=P + 64), dict(refs_out=2 * P - 4)]
    bad += {"fork": [dict(src=None), dict(dst=None), dict(n=0), dict(seq_lens=None)],
            "reserve": [dict(seq_lens=None), dict(new_lens=None), dict(copies=None), dict(max_copies=3), dict(ws=None)],
            "trim": [dict(seq_lens=None), dict(n_sink=-1), dict(window=-1)],
            "compact": [dict(copies=None), dict(max_copies=49), dict(ws=None)]}[name]
    for kw in bad:
        assert blocks(mla, name, **kw) == mla.MLA_ERR_INVALID_ARG, kw
    for kw in (dict(table=P + 2), dict(status=10 * P + 1)):
        assert blocks(mla, name, **kw) == mla.MLA_ERR_ALIGNMENT, kw
    if name in ("reserve", "compact"):
        assert blocks(mla, name, ws_bytes=64) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
        assert blocks(mla, name, ws=P + 4) == mla.MLA_ERR_ALIGNMENT


def test_copy_calls_refuse_bad_arguments(mla):
    cfg = mla.make_config(64, 8, 4, 64, 4, 64)
    ring = mla.make_config(64, 8, 4, 64, 4, 64, cache="int4_g32", resid=128)
    paged = mla.MlaCache(P, None, 2 * P, 2, 256, None, None, 3 * P, 10)
    flat = mla.MlaCache(P, None, 2 * P, 2, 256)
    copy = lambda cfg, c, copies=P, n=4, st=P: mla._lib.mla_blocks_copy(  # noqa: E731
        ctypes.byref(cfg), ctypes.byref(c), copies, n, st, None)
    assert copy(cfg, flat) == mla.MLA_ERR_INVALID_ARG
    assert copy(cfg, paged, None) == copy(cfg, paged, P, 0) == copy(cfg, paged, P, 4, None) == mla.MLA_ERR_INVALID_ARG
    assert copy(ring, paged) == mla.MLA_ERR_INVALID_ARG            # no scales, no ring
    assert copy(cfg, paged, P + 1) == mla.MLA_ERR_ALIGNMENT
    assert mla._lib.mla_blocks_copy(None, ctypes.byref(paged), P, 4, P, None) == mla.MLA_ERR_INVALID_ARG
    rc = lambda cfg, c: mla._lib.mla_ring_copy(ctypes.byref(cfg), ctypes.byref(c), P, P, 1, None, P, None)  # noqa: E731
    assert rc(cfg, flat) == mla.MLA_ERR_INVALID_ARG                # no residual window
    full = mla.MlaCache(P, 2 * P, 3 * P, 2, 256, 4 * P, None)
    assert rc(ring, full) == mla.MLA_ERR_INVALID_ARG


def test_binding_checks_tensors(mla):
    t = torch.zeros(2, 3, dtype=torch.int32)
    r, st = torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # host tensors
        mla.mla_blocks_trim(t, r, r[:2], 0, 4, t, r, st)
    with pytest.raises(ValueError):   # int64 lengths
        mla.mla_blocks_trim(t.long(), r, r[:2], 0, 4, t, r, st)


def test_tokens_without_a_block(mla):
    from mha_mla_latent_b200.cache import LatentCache
    c = LatentCache(mla.make_config(64, 8, 4, 64, 4, 64), 1, 256, "cpu", block_table=[[1, -1]], n_blocks=2)
    c.set_latent_rows(0, 120, torch.ones(8, 64))
    assert c.latent_rows(0, 120, 128).eq(1).all()
    with pytest.raises(ValueError):   # not the pool's last block
        c.latent_rows(0, 120, 129)
    with pytest.raises(ValueError):
        c.set_latent_rows(0, 128, torch.ones(1, 64))


def test_pool_refuses_bad_sizes(mla):
    from mha_mla_latent_b200.cache import BlockPool
    for B, T, n in [(0, 128, 4), (1, 100, 4), (1, 128, 0)]:
        with pytest.raises(ValueError):
            BlockPool(B, T, n, device="cpu")


def test_host_tensors_are_refused(mla):
    """A pointer of a host tensor never reaches the device: every tensor of the window and block
    calls has to be on the current one, the cache's arrays included."""
    cfg = mla.make_config(64, 8, 4, 64, 4, 64)
    plan = mla.Plan(None, cfg)   # refused before the plan is looked at
    cache = mla.cache_struct(torch.zeros(2, 128, 64, dtype=torch.bfloat16), None,
                             torch.zeros(2, 128, 4, 8, dtype=torch.bfloat16), 2, 128)
    lens, ws = torch.ones(2, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_decode_window(plan, cache, lens, q, q, ws, 0, 4)
    q4 = q.unsqueeze(1).expand(2, 3, 8, 64).contiguous()
    with pytest.raises(ValueError):
        mla.mla_decode_chunk_window(plan, cache, lens, q4, q4, ws, 0, 4)
    for wrong in (q4, q[:, :7], q[..., :32]):   # not [B][H][d_h]: a chunk's queries, fewer heads or dims
        with pytest.raises(ValueError, match="q must be"):
            mla.mla_decode_window(plan, cache, lens, wrong, wrong, ws, 0, 4)
    with pytest.raises(ValueError, match="q must be"):
        mla.mla_decode_chunk_window(plan, cache, lens, q, q, ws, 0, 4)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    table, refs, st, cp = i(2, 3), i(5), i(4), i(4, 3)
    for call in (lambda: mla.mla_blocks_copy(cfg, cache, cp, st), lambda: mla.mla_ring_copy(cfg, cache, i(1), i(1), st),
                 lambda: mla.mla_blocks_fork(table, refs, i(1), i(1), i(2), table, refs, st),
                 lambda: mla.mla_blocks_reserve(table, refs, i(2), i(2), table, refs, cp, st, ws),
                 lambda: mla.mla_blocks_compact(table, refs, table, refs, cp, st, ws)):
        with pytest.raises(ValueError):
            call()
    assert cache.device == -1


def test_import_with_a_torch_without_cuda(mla):
    """The entry points that need no GPU work where torch was built without CUDA."""
    import os
    import subprocess
    import sys
    program = ("import torch; del torch._C._cuda_getCurrentRawStream\n"
               "import mha_mla_latent_b200._lib as L\n"
               "cfg = L.make_config(64, 8, 4, 64, 4, 64)\n"
               "print(L.mla_fixed_pairs(cfg, L.MLA_PAIRS_HIGH).tolist(), L.mla_cache_bytes_per_token(cfg))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == "[[0, 1, 2, 3], [0, 1, 2, 3], [0, 1, 2, 3], [0, 1, 2, 3]] 192".split()
