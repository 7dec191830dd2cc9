"""Random latent caches and a plain float64 windowed attention for the window tests.

The reference is the definition: every visible token's key and value are rebuilt from its
latent, nothing is absorbed, nothing is tiled.  It runs on the CPU in float64 and shares no
code with the CUDA path.
"""

import numpy as np
import torch

BLOCK, RING, GROUP = 128, 128, 32


class Layer:
    """Random weights of one converted layer, as the CUDA path stores them."""

    def __init__(self, dtype="bf16", cache="same", H=32, n_kv=32, d_h=128, r=4, d_c=256, seed=0, scale=0.0):
        self.dtype, self.cache, self.H, self.n_kv, self.d_h, self.r, self.d_c = dtype, cache, H, n_kv, d_h, r, d_c
        self.scale = scale
        self.td = torch.float32 if dtype == "f32" else torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        norm = lambda *s: (torch.randn(*s, generator=g) * d_c ** -0.5).to(self.td)  # noqa: E731
        self.W_uk, self.W_uv = norm(n_kv, d_c, d_h - 2 * r), norm(n_kv, d_c, d_h)
        self.pairs = np.sort(np.stack([rng.permutation(d_h // 2)[:r] for _ in range(n_kv)]), 1).astype(np.int32)
        self.g = g

    def config(self, mla):
        kind = {"same": "same", "int4": "int4_g32", "int4_r128": "int4_g32", "int2": "int2_g32"}[self.cache]
        return mla.make_config(64, self.H, self.n_kv, self.d_h, self.r, self.d_c, dtype=self.dtype, cache=kind,
                               resid=RING if self.cache == "int4_r128" else 0, softmax_scale=self.scale)

    def plan(self, mla):
        z = lambda *s: torch.zeros(*s, dtype=self.td)  # noqa: E731
        return mla.mla_plan_create(self.config(mla), z(64, self.d_c), z(64, self.n_kv * self.d_h),
                                   torch.from_numpy(self.pairs), self.W_uk, self.W_uv)

    def sequence(self, L):
        """Stored rows of L tokens: dict of CPU tensors, and the latent values `c` (float64)."""
        kr = torch.randn(L, self.n_kv, 2 * self.r, generator=self.g).to(self.td)
        s = {"kr": kr, "L": L}
        if self.cache == "same":
            s["c_kv"] = torch.randn(L, self.d_c, generator=self.g).to(self.td)
            s["c"] = s["c_kv"].double()
            return s
        bits = 2 if self.cache == "int2" else 4
        top, per = 2 ** (bits - 1) - 1, 8 // bits
        code = torch.randint(-top, top + 1, (L, self.d_c), generator=self.g)
        f = (code % 2 ** bits).view(L, self.d_c // per, per)
        s["c_kv"] = sum(f[..., k] << (bits * k) for k in range(per)).to(torch.uint8)
        s["c_scales"] = (torch.rand(L, self.d_c // GROUP, generator=self.g) * 0.3 + 0.1).to(torch.float16)
        s["c"] = code.double() * s["c_scales"].double().repeat_interleave(GROUP, 1)
        if self.cache == "int4_r128":
            t = torch.arange(max(0, L - RING), L)
            s["ring"] = torch.randn(len(t), self.d_c, generator=self.g).to(self.td)
            s["c"][t] = s["ring"].double()
        return s

    def queries(self, *shape):
        return torch.randn(*shape, self.H, self.d_h, generator=self.g).to(self.td)

    def reference(self, q, seq, p, n_sink, window):
        """q [H][d_h] at position p over the visible tokens of `seq` -> float64 [H][d_h]."""
        t = torch.arange(p + 1)
        t = t[(t < n_sink) | (t > p - window)]
        c, kr, q = seq["c"][t], seq["kr"][t].double(), q.double()
        scale = self.scale or self.d_h ** -0.5
        out = torch.zeros(self.H, self.d_h, dtype=torch.float64)
        for h in range(self.H):
            g = h // (self.H // self.n_kv)
            k = self.pairs[g]
            rope = np.stack([2 * k, 2 * k + 1], -1).reshape(-1)
            nope = np.setdiff1d(np.arange(self.d_h), rope)
            ang = torch.from_numpy(p * 10000.0 ** (-2.0 * k / self.d_h))
            x, y = q[h, 2 * k], q[h, 2 * k + 1]
            rot = torch.stack([x * ang.cos() - y * ang.sin(), x * ang.sin() + y * ang.cos()], -1).reshape(-1)
            s = ((c @ self.W_uk[g].double()) @ q[h, nope] + kr[:, g] @ rot) * scale
            out[h] = torch.softmax(s, 0) @ (c @ self.W_uv[g].double())
        return out


def store(cache, b, seq, hidden=None):
    """Writes a sequence's rows into a LatentCache; the rows of the tokens `hidden` hold NaN."""
    L = seq["L"]
    if L == 0:
        return
    c_kv, kr = seq["c_kv"].clone(), seq["kr"].clone()
    if hidden is not None and len(hidden):
        kr[hidden] = float("nan")
        if c_kv.is_floating_point():
            c_kv[hidden] = float("nan")
    cache.set_latent_rows(b, 0, c_kv)
    if cache.k_rope is not None:
        cache.set_k_rope_tokens(b, 0, kr)
    if cache.c_scales is not None:
        sc = seq["c_scales"].clone()
        if hidden is not None and len(hidden):
            sc[hidden] = float("nan")
        cache.set_scale_rows(b, 0, sc)
    if cache.c_resid is not None:
        t = torch.arange(max(0, L - RING), L)
        cache.c_resid[b, t % RING] = seq["ring"].to(cache.c_resid.device)
        cache.resid_pos[b, t % RING] = t.to(torch.int32).to(cache.resid_pos.device)


def hidden_tokens(L, first_p, n_sink, window):
    """Tokens of [0, L) that no query from position first_p on sees."""
    t = torch.arange(L)
    return t[(t >= n_sink) & (t <= first_p - window)]


def make_cache(mla, layer, B, T_cap, paged, seed=0):
    from mha_mla_latent_b200.cache import LatentCache
    cfg = layer.config(mla)
    if not paged:
        return LatentCache(cfg, B, T_cap, "cuda")
    C = T_cap // BLOCK
    ids = np.random.default_rng(seed).permutation(B * C + 3)[:B * C].reshape(B, C).astype(np.int32)
    return LatentCache(cfg, B, T_cap, "cuda", block_table=ids, n_blocks=B * C + 3)
