"""Decode over layer shapes at the edges of what the CUDA-core kernels take: latents wider than 256
or not a multiple of 16, head dims that are even but not multiples of four."""

import pytest
import torch

from tests.helpers import assert_close
from tests.window_helpers import Layer, hidden_tokens, make_cache, store

pytestmark = pytest.mark.gpu


def check_decode(**kw):
    """mla_decode and mla_decode_window against the definition."""
    import mha_mla_latent_b200 as mla
    layer = Layer(**kw, seed=40)
    lens, T_cap = [200, 1, 77, 130], 256
    seqs = [layer.sequence(L) for L in lens]
    q = layer.queries(len(lens))
    plan = layer.plan(mla)
    L32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, len(lens)), dtype=torch.uint8, device="cuda").fill_(0xFF)
    for kernel in (0, 1):
        if kernel == 1 and layer.H * layer.d_c > 8192:
            continue   # (more than the CUDA-core kernel takes)
        mla.mla_plan_set_option(plan, mla.MLA_OPT_DECODE_KERNEL, kernel)
        for n_sink, window in [(0, 0), (5, 60), (0, 1000)]:   # (0, 0): no window
            cache = make_cache(mla, layer, len(lens), T_cap, True)
            for b, s in enumerate(seqs):
                store(cache, b, s, hidden_tokens(lens[b], lens[b] - 1, n_sink, window) if window else None)
            out = torch.full_like(q, float("nan"), device="cuda")
            if window:
                mla.mla_decode_window(plan, cache.struct, L32, q.cuda(), out, ws, n_sink, window)
            else:
                mla.mla_decode(plan, cache.struct, L32, q.cuda(), out, ws)
            assert mla.mla_device_error(plan) == 0
            for b, L in enumerate(lens):
                ref = layer.reference(q[b], seqs[b], L - 1, n_sink, window or 1000).numpy()
                assert_close(out[b].double().cpu().numpy(), ref, layer.dtype, f"{kw} kernel {kernel} {n_sink} {window} {L}")
    plan.close()


@pytest.mark.parametrize("dtype,H,n_kv,d_h,r,d_c", [("f32", 8, 2, 64, 0, 300), ("f32", 4, 4, 32, 2, 260), ("bf16", 8, 2, 64, 3, 304),
                                                    ("f32", 2, 1, 64, 4, 1020), ("f32", 4, 1, 64, 4, 512)])
def test_latents_wider_than_256(dtype, H, n_kv, d_h, r, d_c):
    """Their last columns are merged by part of a warp."""
    check_decode(dtype=dtype, H=H, n_kv=n_kv, d_h=d_h, r=r, d_c=d_c)


@pytest.mark.parametrize("cache,H,n_kv,d_h,r,d_c", [("int4", 8, 4, 64, 4, 288), ("int2", 4, 1, 64, 3, 320), ("int4_r128", 6, 2, 48, 4, 416),
                                                    ("int4", 8, 8, 30, 1, 1024), ("int4_r128", 2, 2, 128, 0, 512)])
def test_wide_latents_in_groups(cache, H, n_kv, d_h, r, d_c):
    """The same with 4- or 2-bit latents, and with the newest tokens from the ring."""
    check_decode(dtype="bf16", cache=cache, H=H, n_kv=n_kv, d_h=d_h, r=r, d_c=d_c)


@pytest.mark.parametrize("dtype,H,n_kv,d_h,r,d_c", [("f32", 6, 3, 30, 2, 32), ("f32", 4, 4, 18, 4, 20), ("bf16", 4, 2, 22, 3, 64),
                                                    ("bf16", 8, 8, 34, 4, 32), ("f32", 40, 10, 26, 1, 64), ("bf16", 6, 1, 6, 1, 32)])
def test_head_dims_that_are_not_multiples_of_four(dtype, H, n_kv, d_h, r, d_c):
    """The query rows in shared memory start on whole 16 bytes."""
    check_decode(dtype=dtype, H=H, n_kv=n_kv, d_h=d_h, r=r, d_c=d_c)


@pytest.mark.parametrize("H,n_kv,d_h,r,d_c", [(4, 2, 64, 3, 36), (8, 8, 128, 2, 20), (3, 1, 64, 5, 40), (8, 1, 96, 4, 100), (2, 2, 64, 3, 264),
                                              (10, 2, 64, 4, 72)])
def test_bf16_latents_that_are_not_multiples_of_16(H, n_kv, d_h, r, d_c):
    """The merge's product with W_uv takes 16 latent columns a step on the tensor cores, or goes column
    by column."""
    check_decode(dtype="bf16", H=H, n_kv=n_kv, d_h=d_h, r=r, d_c=d_c)


def test_wide_latents_of_many_sequences():
    """The merge takes fewer rows per CTA where the latents leave no room for more."""
    import mha_mla_latent_b200 as mla
    layer = Layer(dtype="f32", H=2, n_kv=1, d_h=32, r=4, d_c=1024, seed=41)
    B = 300
    seq = layer.sequence(40)
    cache = make_cache(mla, layer, B, 40, False)
    for b in range(B):
        store(cache, b, seq)
    plan = layer.plan(mla)
    q = layer.queries(B)
    out = torch.empty_like(q, device="cuda")
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, B), dtype=torch.uint8, device="cuda")
    lens = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    mla.mla_decode(plan, cache.struct, lens, q.cuda(), out, ws)
    assert mla.mla_device_error(plan) == 0
    for b in (0, 151, 299):
        assert_close(out[b].double().cpu().numpy(), layer.reference(q[b], seq, 39, 0, 40).numpy(), "f32", str(b))
    plan.close()


@pytest.mark.parametrize("H,n_kv,d_h,d_c", [(64, 8, 64, 128), (40, 20, 64, 64), (128, 2, 32, 256), (36, 9, 48, 96)])
def test_residual_window_with_more_than_32_heads(H, n_kv, d_h, d_c):
    """The newest 128 tokens come from the ring for every number of heads."""
    check_decode(H=H, n_kv=n_kv, d_h=d_h, r=4, d_c=d_c, cache="int4_r128")
