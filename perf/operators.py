"""Cases of the windowed latent attention and of the cache block operators.

Attention with a sliding window and sinks over the latent cache: the query at position p
attends to the tokens t <= p with t < n_sink or t > p - window.  With the absorbed query
    q_lat[h] = q[h] (NoPE dims) W_uk[g(h)]^T,     q_rope[h] = kept pairs of q[h], rotated at p
    s[h][t]  = (q_lat[h] . c[t] + q_rope[h] . k_rope[t][g(h)]) / sqrt(d_h)
    out[h]   = (softmax over the visible t of s[h]) c W_uv[g(h)]
in its single-token form ("decode") and for the newest Q tokens of each sequence ("chunk").

Cache blocks: a table [B][C] of 128-token pool blocks (-1: none) and a reference count per
block.  "fork": parallel samples share their prompt's blocks (fork), get room for their next
tokens with the shared partial block copied on write (reserve), and the copies are made.
"trim": the blocks that no window reaches any more are released.  "compact": the live blocks
move to the front of the pool and the tables follow.

`own` selects the framework's calls; otherwise everything is elementary torch operations.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
GROUP = 32          # latent values per scale of a quantised cache
RING = 128          # tokens of the unquantised residual window

# Layer shapes of the repository's workloads.
SHAPES = {
    "tiny": dict(dtype="f32", H=4, n_kv=4, d_h=32, r=2, d_c=32),
    "smollm": dict(dtype="bf16", H=9, n_kv=3, d_h=64, r=4, d_c=32),
    "llama": dict(dtype="bf16", H=32, n_kv=32, d_h=128, r=4, d_c=256),
}


def _decode(name, shape, batch, lo, hi, window, n_sink, cache="same", paged=False, d_c=0, queries=1, lens_seed=0):
    c = dict(op="decode" if queries == 1 else "chunk", shape=shape, batch=batch, lo=lo, hi=hi, window=window,
             n_sink=n_sink, cache=cache, paged=paged, d_c=d_c or SHAPES[shape]["d_c"], queries=queries,
             lens_seed=lens_seed)
    return dict(c, name=name) if name else c


def _blocks(name, op, rows, lo, hi, n_blocks, d_c, kids=0, grow=1, window=0, n_sink=0, lens_seed=0):
    c = dict(op=op, rows=rows, lo=lo, hi=hi, n_blocks=n_blocks, d_c=d_c, kids=kids, grow=grow, window=window,
             n_sink=n_sink, lens_seed=lens_seed)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest call: one short float32 sequence, all latency
        _decode("decode_tiny_f32", "tiny", 1, 64, 64, 24, 4),
        # grouped query heads, a small model serving a few sequences
        _decode("decode_smollm_bf16", "smollm", 16, 2048, 2048, 512, 4),
        # the default workload's layer at twice its context, the window its context: the largest bf16 call
        _decode("decode_llama_bf16", "llama", 32, 8192, 8192, 4096, 64),
        # long ragged documents in a paged cache, some of them shorter than the window
        _decode("decode_llama_ragged_paged", "llama", 8, 1024, 32768, 8192, 128, paged=True, d_c=64, lens_seed=3),
        # 4-bit latents, a wide batch, windows that start inside blocks
        _decode("decode_llama_int4_paged", "llama", 64, 7000, 8192, 4001, 4, cache="int4", paged=True, d_c=128,
                lens_seed=4),
        # chunked prefill of prompts: 64 new tokens of each sequence
        _decode("chunk_llama_bf16", "llama", 8, 4096, 4096, 1024, 4, queries=64),
        # a whole odd-sized prompt piece over grouped heads, paged, windows of another size than the blocks
        _decode("chunk_smollm_paged", "smollm", 6, 700, 2048, 500, 7, paged=True, queries=301, lens_seed=5),
        # four samples of each of four prompts, the small pool of a small model
        _blocks("fork_small", "fork", 4, 100, 1000, 256, 32, kids=3, grow=1, lens_seed=6),
        # 32 prompts with four samples each in the default workload's layer
        _blocks("fork_llama", "fork", 32, 1024, 4096, 2048, 256, kids=4, grow=40, lens_seed=7),
        # a wide batch of long sequences slides on
        _blocks("trim_long", "trim", 256, 1024, 32768, 65536, 0, window=4096, n_sink=64, lens_seed=8),
        # a small pool with holes
        _blocks("compact_small", "compact", 12, 100, 2000, 300, 32, lens_seed=9),
        # half of a large pool of the default workload's layer is live, scattered
        _blocks("compact_llama", "compact", 64, 2048, 6144, 4096, 256, lens_seed=10),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["decode", "decode", "decode", "chunk", "chunk", "fork", "trim", "compact"])
    s = rng.randrange(1, 1 << 20)
    if op in ("decode", "chunk"):
        shape = rng.choice(["smollm", "llama", "llama"] + (["tiny"] if op == "decode" else []))
        hi = log(64, 512) if shape == "tiny" else log(512, 16384)
        n_sink, window = rng.choice([0, 1, 4, 64, 100, 128]), log(16, min(hi, 4096))
        paged = rng.random() < 0.5
        d_c, cache = 32, "same"
        if shape == "llama":
            d_c = rng.choice([64, 128, 256])
            cache = rng.choice(["same", "int4", "int2"] + (["int4_r128"] if op == "decode" else []))
        if op == "decode":
            batch = log(1, 4) if shape == "tiny" else log(1, 48)
            return _decode(None, shape, batch, max(1, hi // 4), hi, window, n_sink, cache, paged, d_c, 1, s)
        queries = log(2, 200)
        window = min(window, 1024)
        return _decode(None, shape, log(1, 6), max(queries, hi // 4), max(queries, min(hi, 4096)), window, n_sink,
                       cache, paged, d_c, queries, s)
    d_c = rng.choice([32, 64, 256])
    if op == "fork":
        rows, kids, hi = log(1, 24), rng.randrange(1, 5), log(128, 4096)
        need = rows * (-(-hi // BLOCK) + (kids + 1) * 3)
        return _blocks(None, "fork", rows, max(1, hi // 4), hi, need + rng.randrange(8), d_c, kids,
                       rng.choice([1, 7, 130, 200]), 0, 0, s)
    rows, hi = log(1, 64), log(128, 4096 if op == "compact" else 32768)
    need = rows * -(-hi // BLOCK)
    if op == "compact":
        return _blocks(None, "compact", rows, max(1, hi // 4), hi, need + log(1, need + 1), d_c, 0, 1, 0, 0, s)
    return _blocks(None, "trim", rows, max(1, hi // 8), hi, need + rng.randrange(64), 0, 0, 1, log(1, 8192),
                   rng.choice([0, 1, 64, 300]), s)


# ------------------------------------------------------------------ sizes
def _lens(case):
    n = case["batch"] if "batch" in case else case["rows"]
    return np.random.default_rng([17, case["lens_seed"]]).integers(case["lo"], case["hi"] + 1, size=n)


def _row_bytes(cache, d_c, R, eb):
    if cache == "same":
        return d_c * eb + R * eb
    return d_c * (2 if cache == "int2" else 4) // 8 + d_c // GROUP * 2 + R * eb


def work(case):
    lens = _lens(case)
    if case["op"] in ("decode", "chunk"):
        sh, d_c, Q = SHAPES[case["shape"]], case["d_c"], case["queries"]
        H, n_kv, d_h, r = sh["H"], sh["n_kv"], sh["d_h"], sh["r"]
        R, eb = n_kv * 2 * r, 4 if sh["dtype"] == "f32" else 2
        S, W = case["n_sink"], case["window"]
        union = pairs = 0
        for L in lens.tolist():
            p = np.arange(L - Q, L)
            pairs += int((np.minimum(S, np.maximum(p - W + 1, 0)) + np.minimum(W, p + 1)).sum())
            lo = max(0, L - Q - W + 1)
            union += (L - lo) + min(S, lo)
        n_q = len(lens) * Q * H
        weights = n_kv * (d_c * (d_h - 2 * r) + d_c * d_h) * eb
        return {"bytes": union * _row_bytes(case["cache"], d_c, R, eb) + weights + 2 * n_q * d_h * eb,
                "flops": 2 * pairs * H * (2 * d_c + 2 * r) + 2 * n_q * d_c * (2 * d_h - 2 * r)}
    cols = -(-(case["hi"] + case["grow"]) // BLOCK)
    rows = case["rows"] * (1 + case["kids"])
    control = 2 * 4 * (rows * cols + case["n_blocks"])
    row = (case["d_c"] + _R(case)) * 2
    if case["op"] == "fork":
        return {"bytes": control + 2 * case["kids"] * int((lens % BLOCK).sum()) * row, "flops": 0}
    if case["op"] == "trim":
        return {"bytes": control, "flops": 0}
    live = int((-(-lens // BLOCK)).sum())   # a random half of the pool's ids below `live` is free: that many blocks move
    moves = live * (case["n_blocks"] - live) // case["n_blocks"]
    return {"bytes": control + 2 * moves * BLOCK * row, "flops": 0}


def _R(case):   # RoPE key values per token: 32 KV heads x 8 dims, or the small model's 3 x 8
    return 24 if case["d_c"] == 32 else 256


# ------------------------------------------------------------------ inputs
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    return _prepare_attention(case, g, rng) if case["op"] in ("decode", "chunk") else _prepare_blocks(case, g, rng)


def _prepare_attention(case, g, rng):
    sh = SHAPES[case["shape"]]
    H, n_kv, d_h, r, d_c = sh["H"], sh["n_kv"], sh["d_h"], sh["r"], case["d_c"]
    dt = torch.float32 if sh["dtype"] == "f32" else torch.bfloat16
    B, Q, lens = case["batch"], case["queries"], _lens(case)
    T_cap = -(-int(lens.max()) // BLOCK) * BLOCK
    C = T_cap // BLOCK
    if case["paged"]:
        n_blocks = B * C + 5
        table = torch.from_numpy(rng.permutation(n_blocks)[:B * C].reshape(B, C).astype(np.int32)).cuda()
        rows, cap = n_blocks, BLOCK
    else:
        n_blocks, table, rows, cap = 0, None, B, T_cap
    c_scales = c_resid = resid_pos = None
    if case["cache"] == "same":
        c_kv = _normal(g, (rows, cap, d_c), dt)
    else:   # random codes; the scales of values of about unit size
        bits = 2 if case["cache"] == "int2" else 4
        top = 2 ** (bits - 1) - 1
        codes = torch.randint(-top, top + 1, (rows, cap, d_c), generator=g, device="cuda", dtype=torch.int32)
        per = 8 // bits
        field = (codes & (2 ** bits - 1)).view(rows, cap, d_c // per, per)
        c_kv = (field << (bits * torch.arange(per, device="cuda", dtype=torch.int32))).sum(-1).to(torch.uint8)
        c_scales = (torch.rand((rows, cap, d_c // GROUP), generator=g, device="cuda") * 0.3 + 0.1).to(torch.float16)
        if case["cache"] == "int4_r128":   # the newest 128 tokens of each sequence, unquantised
            c_resid = _normal(g, (B, RING, d_c), dt)
            resid_pos = np.full((B, RING), -1, dtype=np.int32)
            for b, L in enumerate(lens.tolist()):
                t = np.arange(max(0, L - RING), L)
                resid_pos[b, t % RING] = t
            resid_pos = torch.from_numpy(resid_pos).cuda()
    st = dict(case=dict(case), c_kv=c_kv, c_scales=c_scales, c_resid=c_resid, resid_pos=resid_pos, table=table,
              n_blocks=n_blocks, T_cap=T_cap,
              k_rope=_normal(g, (rows, cap, n_kv, 2 * r), dt),
              lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
              q=_normal(g, (B, Q, H, d_h), dt),
              W_uk=_normal(g, (n_kv, d_c, d_h - 2 * r), dt, d_c ** -0.5),
              W_uv=_normal(g, (n_kv, d_c, d_h), dt, d_c ** -0.5),
              pairs=np.sort(np.stack([rng.permutation(d_h // 2)[:r] for _ in range(n_kv)]), axis=1).astype(np.int32))
    rope, nope = _dims(st["pairs"], d_h)
    st["rope_dims"], st["nope_dims"] = torch.from_numpy(rope).cuda(), torch.from_numpy(nope).cuda()
    st["theta"] = 10000.0 ** (-2.0 * torch.from_numpy(st["pairs"]).cuda().double() / d_h)   # [n_kv][r]
    if own:
        _prepare_own(st, sh, d_c)
    return st


def _dims(pairs, d_h):
    """The kept (RoPE) and the other (NoPE) dims of each KV head, ascending."""
    rope = np.stack([2 * pairs, 2 * pairs + 1], axis=-1).reshape(pairs.shape[0], -1).astype(np.int64)
    nope = np.stack([np.setdiff1d(np.arange(d_h), row) for row in rope])
    return rope, nope


def _prepare_own(st, sh, d_c):
    """The plan, the cache view, the workspace and the output that a serving program keeps."""
    import mha_mla_latent_b200 as mla
    kind = st["case"]["cache"]
    hidden = 64   # the attention does not see the hidden size; the append weights are not used here
    cfg = mla.make_config(hidden, sh["H"], sh["n_kv"], sh["d_h"], sh["r"], d_c, dtype=sh["dtype"],
                          cache="same" if kind == "same" else "int2_g32" if kind == "int2" else "int4_g32",
                          resid=RING if kind == "int4_r128" else 0)
    dt = st["q"].dtype
    st["plan"] = mla.mla_plan_create(cfg, torch.zeros(hidden, d_c, dtype=dt),
                                     torch.zeros(hidden, sh["n_kv"] * sh["d_h"], dtype=dt),
                                     torch.from_numpy(st["pairs"]), st["W_uk"].cpu(), st["W_uv"].cpu())
    B, Q = st["case"]["batch"], st["case"]["queries"]
    st["cache"] = mla.cache_struct(st["c_kv"], st["c_scales"], st["k_rope"], B, st["T_cap"], st["c_resid"],
                                   st["resid_pos"], st["table"], st["n_blocks"])
    n = mla.mla_decode_workspace_bytes(st["plan"], B) if Q == 1 else \
        mla.mla_decode_chunk_workspace_bytes(st["plan"], B, Q)
    st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    st["out"] = torch.empty_like(st["q"])


def _prepare_blocks(case, g, rng):
    lens, n_blocks, d_c, R = _lens(case), case["n_blocks"], case["d_c"], _R(case)
    rows = case["rows"] * (1 + case["kids"])
    C = -(-(case["hi"] + case["grow"]) // BLOCK)
    table = np.full((rows, C), -1, dtype=np.int32)
    ids, at = rng.permutation(n_blocks).astype(np.int32), 0
    for b, L in enumerate(lens.tolist()):
        k = -(-L // BLOCK)
        shared = min(k // 2, -(-int(lens[b - 1]) // BLOCK)) if case["op"] == "trim" and b % 2 else 0
        table[b, :shared] = table[b - 1, :shared]          # a common prefix with the row before
        table[b, shared:k] = ids[at:at + k - shared]
        at += k - shared
    refs = np.bincount(table[table >= 0], minlength=n_blocks).astype(np.int32)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    st = dict(case=dict(case), table=up(table), refs=up(refs), lens=up(np.concatenate([lens] * (1 + case["kids"]))))
    st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
    if case["op"] != "trim":
        st["c_kv"] = _normal(g, (n_blocks, BLOCK, d_c), torch.bfloat16)
        st["k_rope"] = _normal(g, (n_blocks, BLOCK, R // 8, 8), torch.bfloat16)
    if case["op"] == "fork":
        n = case["rows"]
        st["src"] = up(np.concatenate([np.arange(n)] * case["kids"]))
        st["dst"] = up(np.arange(n, rows))
        st["new_lens"] = up(np.concatenate([lens] * (1 + case["kids"])) + rng.integers(1, case["grow"] + 1, size=rows))
    if own:
        import mha_mla_latent_b200 as mla
        st["status"] = torch.zeros(mla.MLA_BLOCKS_STATUS_INTS, dtype=torch.int32, device="cuda")
        st["ws"] = torch.empty(mla.mla_blocks_workspace_bytes(rows, C, n_blocks), dtype=torch.uint8, device="cuda")
        if case["op"] != "trim":
            st["copies"] = torch.empty(max(rows, n_blocks // 2, 1), 3, dtype=torch.int32, device="cuda")
            st["cfg"] = mla.make_config(64, R // 8, R // 8, 64, 4, d_c)
            st["cache"] = mla.cache_struct(st["c_kv"], None, st["k_rope"], rows, C * BLOCK, block_table=st["table_out"],
                                           n_blocks=n_blocks)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op in ("decode", "chunk"):
        return _attention(st)
    return {"fork": _fork, "trim": _trim, "compact": _compact}[op](st)


def _run_own(st, op):
    import mha_mla_latent_b200 as mla
    case = st["case"]
    if op == "decode":
        B, _, H, d_h = st["q"].shape
        mla.mla_decode_window(st["plan"], st["cache"], st["lens"], st["q"].view(B, H, d_h), st["out"].view(B, H, d_h),
                              st["ws"], case["n_sink"], case["window"])
        return st["out"]
    if op == "chunk":
        mla.mla_decode_chunk_window(st["plan"], st["cache"], st["lens"], st["q"], st["out"], st["ws"], case["n_sink"],
                                    case["window"])
        return st["out"]
    table, refs = st["table_out"], st["refs_out"]
    if op == "trim":
        mla.mla_blocks_trim(st["table"], st["refs"], st["lens"], case["n_sink"], case["window"], table, refs,
                            st["status"])
        return table, refs
    if op == "fork":
        mla.mla_blocks_fork(st["table"], st["refs"], st["src"], st["dst"], st["lens"], table, refs, st["status"])
        mla.mla_blocks_reserve(table, refs, st["lens"], st["new_lens"], table, refs, st["copies"], st["status"], st["ws"])
    else:
        mla.mla_blocks_compact(st["table"], st["refs"], table, refs, st["copies"], st["status"], st["ws"])
    mla.mla_blocks_copy(st["cfg"], st["cache"], st["copies"], st["status"])
    return table, refs, st["c_kv"], st["k_rope"]


# ------------------------------------------------------------------ plain attention
def _latent(st, slot, b, t):
    """float32 latent rows of tokens t [B][N] of sequences b [B][1] at flat cache rows `slot`."""
    case, d_c = st["case"], st["case"]["d_c"]
    flat = st["c_kv"].view(-1, st["c_kv"].shape[-1])[slot]
    if case["cache"] == "same":
        return flat.float()
    bits = 2 if case["cache"] == "int2" else 4
    per, half = 8 // bits, 2 ** (bits - 1)
    f = (flat.int().unsqueeze(-1) >> (bits * torch.arange(per, device=flat.device, dtype=torch.int32))) & (2 * half - 1)
    code = ((f ^ half) - half).view(*flat.shape[:-1], d_c // GROUP, GROUP)
    scale = st["c_scales"].view(-1, d_c // GROUP)[slot].float()
    c = (code.float() * scale.unsqueeze(-1)).view(*flat.shape[:-1], d_c)
    if st["c_resid"] is not None:
        ring = t % RING
        new = (t >= st["lens"].long()[:, None] - RING) & (st["resid_pos"][b, ring] == t)
        c = torch.where(new.unsqueeze(-1), st["c_resid"][b, ring].float(), c)
    return c


def _attention(st):
    case, q = st["case"], st["q"].float()
    B, Q, H, d_h = q.shape
    n_kv, r2, d_c, S, W = st["W_uk"].shape[0], st["k_rope"].shape[-1], case["d_c"], case["n_sink"], case["window"]
    dev, G = q.device, H // n_kv
    L = st["lens"].long()
    p = L[:, None] - Q + torch.arange(Q, device=dev)                         # [B][Q]
    # the tokens any query of the sequence may see: the sinks, then the windows' union
    lo = torch.clamp(L - Q - W + 1, min=S)
    n = min(S + W + Q - 1, st["T_cap"] + S)
    j = torch.arange(n, device=dev)
    t = torch.where(j < S, j, lo[:, None] + (j - S))                          # [B][n]
    inside = t < L[:, None]
    tc = torch.where(inside, t, 0)
    b = torch.arange(B, device=dev)[:, None]
    if st["table"] is not None:
        slot = st["table"].long()[b, tc // BLOCK] * BLOCK + tc % BLOCK
    else:
        slot = b * st["T_cap"] + tc
    c = _latent(st, slot, b, tc)                                              # [B][n][d_c]
    kr = st["k_rope"].view(-1, n_kv, r2)[slot].float()                        # [B][n][n_kv][2r]
    # absorbed NoPE query and rotated RoPE query (angles in 64 bits: positions are large)
    qg = q.view(B, Q, n_kv, G, d_h)
    nope = torch.gather(qg, 4, st["nope_dims"].view(1, 1, n_kv, 1, -1).expand(B, Q, n_kv, G, -1))
    rope = torch.gather(qg, 4, st["rope_dims"].view(1, 1, n_kv, 1, -1).expand(B, Q, n_kv, G, -1))
    q_lat = torch.einsum("bigkd,gcd->bigkc", nope, st["W_uk"].float())
    ang = p[:, :, None, None, None].double() * st["theta"].view(1, 1, n_kv, 1, -1)
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    x, y = rope[..., 0::2], rope[..., 1::2]
    q_rot = torch.stack([x * cos - y * sin, x * sin + y * cos], dim=-1).flatten(-2)
    s = torch.einsum("bigkc,bnc->bigkn", q_lat, c) + torch.einsum("bigkj,bngj->bigkn", q_rot, kr)
    s = s / math.sqrt(d_h)
    seen = inside[:, None] & (t[:, None] <= p[:, :, None]) & ((t[:, None] < S) | (t[:, None] > p[:, :, None] - W))
    s = torch.where(seen[:, :, None, None], s, -math.inf)
    m = torch.clamp(s.amax(-1, keepdim=True), min=-1e30)
    e = torch.exp(s - m)
    o = torch.einsum("bigkn,bnc->bigkc", e, c) / torch.clamp(e.sum(-1, keepdim=True), min=1e-30)
    out = torch.einsum("bigkc,gcd->bigkd", o, st["W_uv"].float())
    return out.reshape(B, Q, H, d_h).to(st["q"].dtype)


# ------------------------------------------------------------------ plain block operators
def _counts(table, n_blocks):
    """How many entries of the table name each block."""
    flat = torch.where(table >= 0, table, n_blocks).long().flatten()
    return torch.zeros(n_blocks + 1, dtype=torch.int32, device=table.device).index_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32))[:n_blocks]


def _fork(st):
    table, refs, lens = st["table"].clone(), st["refs"], st["lens"].long()
    rows, C = table.shape
    col = torch.arange(C, device=table.device)
    # fork: the first ceil(L / 128) entries of the source row
    src, dst = st["src"].long(), st["dst"].long()
    old = table[dst]
    new = torch.where(col < (-(-lens[src] // BLOCK))[:, None], table[src], -1)
    refs = refs + _counts(new, refs.numel()) - _counts(old, refs.numel())
    table[dst] = new
    # reserve: columns without a block that tokens [L, N) touch, and shared partial blocks
    N = st["new_lens"].long()
    first, last = -(-lens // BLOCK), -(-N // BLOCK)
    need = (col >= first[:, None]) & (col < last[:, None]) & (table < 0)
    part = torch.clamp(lens // BLOCK, max=C - 1)
    held = table.gather(1, part[:, None])[:, 0].long()
    write = (lens % BLOCK > 0) & (N > lens) & (held >= 0)
    same = (held[:, None] == held[None, :]) & write[:, None] & write[None, :]
    rank = torch.tril(same, -1).sum(1)          # earlier rows that write into the same block
    cow = write & (refs[held.clamp(min=0)] - rank > 1)
    need |= cow[:, None] & (col == part[:, None])
    order = torch.argsort((refs > 0).int(), stable=True).to(torch.int32)   # free blocks first, lowest ids first
    nth = torch.cumsum(need.flatten().int(), 0) - 1
    got = torch.where(need, order[nth.clamp(min=0)].view(rows, C), table)
    refs = refs + _counts(torch.where(need, got, -1), refs.numel()) - \
        _counts(torch.where(cow, held.int(), -1), refs.numel())
    # the copies: rows [0, L % 128) of the shared block (a row without a copy rewrites the values of a block in use)
    frm = torch.where(held >= 0, held, table[0, 0].long())
    to = torch.where(cow, got.gather(1, part[:, None])[:, 0].long(), frm)
    keep = (torch.arange(BLOCK, device=table.device) < (lens % BLOCK)[:, None]) & cow[:, None]
    values = [torch.where(keep.view(rows, BLOCK, *[1] * (a.dim() - 2)), a[frm], a[to]) for a in (st["c_kv"], st["k_rope"])]
    st["c_kv"][to], st["k_rope"][to] = values
    return got, refs, st["c_kv"], st["k_rope"]


def _trim(st):
    table, lens, case = st["table"], st["lens"].long()[:, None], st["case"]
    t0 = torch.arange(table.shape[1], device=table.device) * BLOCK
    sink = t0 < torch.clamp(lens, max=case["n_sink"])
    kept = sink | ((t0 < lens) & (t0 + BLOCK > lens - case["window"]) & (case["window"] > 0))
    out = torch.where(kept, table, -1)
    return out, st["refs"] + _counts(out, st["refs"].numel()) - _counts(table, st["refs"].numel())


def _compact(st):
    table, refs = st["table"], st["refs"]
    n = refs.numel()
    ids = torch.arange(n, device=refs.device)
    used = refs > 0
    live = used.sum()
    moves, holes = used & (ids >= live), ~used & (ids < live)
    # the i-th live block behind the border moves to the i-th hole before it
    hole = torch.argsort((~holes).int(), stable=True)
    to = torch.where(moves, hole[(torch.cumsum(moves.int(), 0) - 1).clamp(min=0)], ids)
    out = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1)
    # where each block's rows come from: entry n of the longer array takes what does not move
    frm = torch.arange(n + 1, device=refs.device).index_copy_(0, torch.where(moves, to, n), ids)[:n]
    refs_out = torch.where(ids < live, refs[frm], 0)
    for a in (st["c_kv"], st["k_rope"]):
        a.copy_(a[frm])
    return out, refs_out, st["c_kv"], st["k_rope"]


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    """out from the definition in float64, without absorption: every visible token's key and
    value of every head are rebuilt from its latent.  The block operators' outputs are whole
    numbers and moved values: None."""
    if case["op"] not in ("decode", "chunk"):
        return None
    st = prepare(case, seed)
    d_h, d_c, W, S = SHAPES[case["shape"]]["d_h"], case["d_c"], case["window"], case["n_sink"]
    n_kv = st["W_uk"].shape[0]
    q, lens = st["q"].double(), st["lens"].tolist()
    B, Q, H = q.shape[:3]
    uk, uv = st["W_uk"].double(), st["W_uv"].double()
    out = torch.zeros_like(q)
    rope, nope = st["rope_dims"], st["nope_dims"]
    theta = 10000.0 ** (-2.0 * torch.from_numpy(st["pairs"]).double().cuda() / d_h)
    for b, L in enumerate(lens):
        lo = max(0, L - Q - W + 1)
        t = torch.cat([torch.arange(min(S, lo)), torch.arange(lo, L)]).cuda()
        if st["table"] is None:
            place = (torch.full_like(t, b), t)
        else:
            place = (st["table"][b].long()[t // BLOCK], t % BLOCK)
        raw, kr = st["c_kv"][place], st["k_rope"][place].double()
        if case["cache"] == "same":
            c = raw.double()
        else:
            bits = 2 if case["cache"] == "int2" else 4
            fields = [(raw.long() >> (bits * k)) % 2 ** bits for k in range(8 // bits)]
            v = torch.stack(fields, -1).reshape(len(t), d_c)
            v = torch.where(v >= 2 ** (bits - 1), v - 2 ** bits, v).double()
            c = v * st["c_scales"][place].double().repeat_interleave(GROUP, dim=-1)
            if st["c_resid"] is not None:
                newest = t >= L - RING
                c[newest] = st["c_resid"][b][t[newest] % RING].double()
        K = torch.zeros(len(t), n_kv, d_h, dtype=torch.float64, device="cuda")
        K.scatter_(2, nope[None].expand(len(t), -1, -1), torch.einsum("tc,gcd->tgd", c, uk))
        V = torch.einsum("tc,gcd->tgd", c, uv)
        K.scatter_(2, rope[None].expand(len(t), -1, -1), kr)
        pos = torch.arange(L - Q, L, device="cuda")
        ang = pos[:, None, None].double() * theta
        for g in range(n_kv):
            x = q[b][:, g * (H // n_kv):(g + 1) * (H // n_kv)].clone()          # [Q][G][d_h]
            even, odd = x[..., rope[g][0::2]], x[..., rope[g][1::2]]
            cs, sn = ang[:, g].cos()[:, None], ang[:, g].sin()[:, None]
            x[..., rope[g][0::2]] = even * cs - odd * sn
            x[..., rope[g][1::2]] = even * sn + odd * cs
            s = torch.einsum("ikd,td->ikt", x, K[:, g]) / math.sqrt(d_h)
            see = (t[None] <= pos[:, None]) & ((t[None] < S) | (t[None] > pos[:, None] - W))
            a = torch.softmax(s.masked_fill(~see[:, None], -math.inf), dim=-1)
            out[b][:, g * (H // n_kv):(g + 1) * (H // n_kv)] = torch.einsum("ikt,td->ikd", a, V[:, g])
    return out
