"""The block operators against a sequential model in plain Python (whole numbers: equal), the
rows they move (bit for bit), and a serving run that uses them with the windowed attention."""

import numpy as np
import pytest
import torch

from tests.helpers import assert_close
from tests.window_helpers import BLOCK, Layer

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the model
def blocks_of(L):
    return -(-L // BLOCK)


def m_fork(table, refs, src, dst, lens):
    B, C = table.shape
    old, out, refs, err = table, table.copy(), refs.copy(), 0
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (0 <= s < B and 0 <= d < B) or d in dst[:i] or \
                (s != d and any(dj == s and sj != s for sj, dj in zip(src, dst))):
            err |= 32
            continue
        if not 0 <= lens[s] <= C * BLOCK:
            err |= 1
            continue
        k = blocks_of(lens[s])
        for e in old[d][old[d] >= 0]:
            refs[e] -= 1
        for e in old[s][:k][old[s][:k] >= 0]:
            refs[e] += 1
        out[d] = -1
        out[d][:k] = old[s][:k]
    return out, refs, err


def m_reserve(table, refs, lens, new):
    B, C = table.shape
    out, cnt, copies, err = table.copy(), refs.copy(), [], 0
    free = [i for i in range(len(refs)) if refs[i] <= 0]
    n0 = len(free)
    for b in range(B):
        L, N = int(lens[b]), int(new[b])
        if not 0 <= L <= N <= C * BLOCK:
            err |= 1
            continue
        if L % BLOCK and N > L:
            e = out[b][L // BLOCK]
            if e < 0:
                err |= 8
            elif cnt[e] > 1:
                cnt[e] -= 1
                if not free:
                    return table, refs, [], err | 16, 0
                out[b][L // BLOCK] = free.pop(0)
                copies.append((e, out[b][L // BLOCK], L % BLOCK))
                cnt[out[b][L // BLOCK]] = 1
        for j in range(blocks_of(L), blocks_of(N)):
            if out[b][j] < 0:
                if not free:
                    return table, refs, [], err | 16, 0
                out[b][j] = free.pop(0)
                cnt[out[b][j]] = 1
    return out, cnt, copies, err, n0 - len(free)


def m_trim(table, refs, lens, n_sink, window):
    out, refs = table.copy(), refs.copy()
    for b, L in enumerate(lens):
        t = np.arange(L)
        kept = set((t[(t < n_sink) | (t >= L - window)] // BLOCK).tolist())
        for j in range(table.shape[1]):
            if j not in kept and out[b][j] >= 0:
                refs[out[b][j]] -= 1
                out[b][j] = -1
    return out, refs


def m_compact(table, refs):
    n, live = len(refs), int((refs > 0).sum())
    holes = [i for i in range(live) if refs[i] <= 0]
    movers = [i for i in range(live, n) if refs[i] > 0]
    to = dict(zip(movers, holes))
    out = np.vectorize(lambda e: to.get(e, e) if e >= 0 else -1)(table).astype(np.int32)
    cnt = np.zeros_like(refs)
    for i in range(n):
        if refs[i] > 0:
            cnt[to.get(i, i)] = refs[i]
    return out, cnt, [(m, to[m], BLOCK) for m in movers]


# ------------------------------------------------------------------ running the operators
class Dev:
    def __init__(self, table, refs):
        import mha_mla_latent_b200 as mla
        self.mla = mla
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.up, self.table, self.refs = up, up(table), up(refs)
        B, C = table.shape
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.copies = torch.full((max(B, len(refs) // 2, 1), 3), -7, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(mla.mla_blocks_workspace_bytes(B, C, len(refs)), dtype=torch.uint8, device="cuda")
        self.ws.fill_(0x5A)

    def call(self, name, *args, inplace):
        t, r = (self.table, self.refs) if inplace else (torch.full_like(self.table, -9), torch.full_like(self.refs, -9))
        was = None if inplace else (self.table.clone(), self.refs.clone())
        extra = {"fork": (t, r, self.status), "trim": (t, r, self.status),
                 "reserve": (t, r, self.copies, self.status, self.ws),
                 "compact": (t, r, self.copies, self.status, self.ws)}[name]
        getattr(self.mla, "mla_blocks_" + name)(self.table, self.refs, *args, *extra)
        torch.cuda.synchronize()
        if was:   # the input is left as it was
            assert torch.equal(was[0], self.table) and torch.equal(was[1], self.refs)
        self.table, self.refs = t, r
        return t.cpu().numpy(), r.cpu().numpy(), self.status.cpu().numpy()

    def listed(self, n):
        return [tuple(x) for x in self.copies[:n].cpu().tolist()]


def random_state(rng, B, C, n_blocks, share=0.5, holes=0.1):
    """A table with shared prefixes and trimmed entries, its counts, and the lengths."""
    lens = rng.integers(0, C * BLOCK + 1, size=B)
    table = np.full((B, C), -1, dtype=np.int32)
    ids, at = rng.permutation(n_blocks), 0
    for b, L in enumerate(lens):
        k, shared = blocks_of(L), 0
        if b and rng.random() < share:
            o = int(rng.integers(b))
            shared = int(min(k, blocks_of(lens[o])))
            table[b, :shared] = table[o, :shared]
        k = min(k, shared + n_blocks - at)
        lens[b] = min(L, k * BLOCK)
        table[b, shared:k] = ids[at:at + k - shared]
        at += k - shared
        gone = rng.random(C) < holes
        if lens[b]:
            gone[blocks_of(lens[b]) - 1] = False
        table[b, gone] = -1
    refs = np.bincount(table[table >= 0], minlength=n_blocks).astype(np.int32)
    return table, refs, lens.astype(np.int32)


SIZES = [(1, 1, 1), (3, 4, 20), (16, 9, 200), (40, 33, 5000), (1500, 3, 70000), (2, 700, 1500)]


@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("size", SIZES, ids=[str(s) for s in SIZES])
def test_operators_match_the_model(size, inplace):
    B, C, n_blocks = size
    rng = np.random.default_rng(B * 7 + C)
    for trial in range(3):
        table, refs, lens = random_state(rng, B, C, n_blocks)
        d = Dev(table, refs)
        # reserve: short and long growth, some sequences without
        new = np.minimum(lens + rng.choice([0, 1, 5, 129, 2000], size=B), C * BLOCK).astype(np.int32)
        want = m_reserve(table, refs, lens, new)
        got = d.call("reserve", d.up(lens), d.up(new), inplace=inplace)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert got[2].tolist() == [len(want[2]), want[3], int((want[1] > 0).sum()), want[4]]
        assert d.listed(len(want[2])) == want[2]
        # trim
        table, refs = want[:2]
        n_sink, window = [(0, 0), (1, 128), (200, 77)][trial]
        want = m_trim(table, refs, lens, n_sink, window)
        d.status.zero_()
        got = d.call("trim", d.up(lens), n_sink, window, inplace=inplace)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2][1] == 0
        # fork, with pairs to skip among them
        table, refs = want
        n = max(1, B // 2)
        src, dst = rng.integers(0, B, size=n).astype(np.int32), rng.integers(0, B, size=n).astype(np.int32)
        src[rng.random(n) < 0.1], dst[rng.random(n) < 0.1] = B, -1
        flens = lens.copy()
        flens[rng.random(B) < 0.1] = C * BLOCK + 1
        want = m_fork(table, refs, src.tolist(), dst.tolist(), flens.tolist())
        got = d.call("fork", d.up(src), d.up(dst), d.up(flens), inplace=inplace)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2][1] == want[2]
        # compact
        table, refs = want[:2]
        want = m_compact(table, refs)
        d.status.zero_()
        got = d.call("compact", inplace=inplace)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert got[2].tolist() == [len(want[2]), 0, int((refs > 0).sum()), len(want[2])]
        assert d.listed(len(want[2])) == want[2]


def test_copy_on_write_order():
    """Holders of one partly filled block: all but the last writer copy; with a holder that does
    not write, or one outside the table, every writer copies."""
    table = np.array([[0, 3], [0, 3], [0, 3], [0, 3]], dtype=np.int32)
    lens = np.full(4, 130, dtype=np.int32)
    for extra, new, want_copies in [(0, [131] * 4, [0, 1, 2]), (1, [131] * 4, [0, 1, 2, 3]),
                                    (0, [131, 130, 131, 131], [0, 2, 3]), (0, [130, 130, 140, 130], [2])]:
        refs = np.zeros(12, dtype=np.int32)
        refs[0], refs[3] = 4, 4 + extra
        want = m_reserve(table, refs, lens, new)
        d = Dev(table, refs)
        got = d.call("reserve", d.up(lens), d.up(np.array(new)), inplace=True)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert [b for b in range(4) if got[0][b, 1] != 3] == want_copies
        assert d.listed(len(want_copies)) == want[2]


def test_pool_exhausted_changes_nothing():
    table = np.array([[0, -1], [1, -1]], dtype=np.int32)
    refs = np.array([1, 1, 0], dtype=np.int32)
    d = Dev(table, refs)
    got = d.call("reserve", d.up([100, 128]), d.up([200, 129]), inplace=True)   # two blocks wanted, one free
    assert np.array_equal(got[0], table) and np.array_equal(got[1], refs)
    assert got[2].tolist() == [0, d.mla.MLA_DEVERR_POOL, 2, 0]
    # the bit stays until the caller clears it
    got = d.call("reserve", d.up([100, 128]), d.up([128, 129]), inplace=True)
    assert got[2].tolist() == [0, d.mla.MLA_DEVERR_POOL, 3, 1] and got[0][1, 1] == 2


def test_bad_entries_and_lengths_are_flagged():
    table = np.array([[5, 99], [-3, 1], [2, -1]], dtype=np.int32)
    refs = np.array([0, 1, 1, 0, 0, 1, 0, 0], dtype=np.int32)
    d = Dev(table, refs)
    got = d.call("trim", d.up([0, 300, 10]), 0, 0, inplace=False)
    assert got[2][1] == d.mla.MLA_DEVERR_BLOCK | d.mla.MLA_DEVERR_SEQ_LEN
    assert got[0].tolist() == [[-1, -1], [-3, 1], [-1, -1]] and got[1].tolist() == [0, 1, 0, 0, 0, 0, 0, 0]
    d = Dev(table, refs)
    got = d.call("reserve", d.up([10, 5, 200]), d.up([9, 6, 201]), inplace=False)   # N < L; both partial blocks missing
    assert got[2][1] == d.mla.MLA_DEVERR_SEQ_LEN | d.mla.MLA_DEVERR_BLOCK
    assert np.array_equal(got[0], table) and got[2][0] == 0


KINDS = [dict(d_c=256), dict(d_c=128, cache="int4"), dict(d_c=64, cache="int2"), dict(H=4, n_kv=4, d_h=32, d_c=36),
         dict(dtype="f32", H=3, n_kv=1, d_h=20, r=5, d_c=20), dict(H=9, n_kv=3, d_h=64, r=1, d_c=32, cache="int2"),
         dict(H=8, n_kv=8, d_h=32, r=0, d_c=32)]


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_copy_moves_the_listed_rows_only(kind):
    """Every array of a layer's cache, bit for bit; rows behind the copied ones, other blocks
    and entries to be skipped stay as they are."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import LatentCache
    layer = Layer(**kind, seed=1)
    n_blocks = 30
    cache = LatentCache(layer.config(mla), 2, 256, "cuda", block_table=np.zeros((2, 2), dtype=np.int32), n_blocks=n_blocks)
    arrays = [a for a in (cache.c_kv, cache.c_scales, cache.k_rope) if a is not None]
    for a in arrays:
        raw = torch.randint(0, 256, (a.numel() * a.element_size(),), dtype=torch.uint8, device="cuda")
        a.view(torch.uint8).view(-1).copy_(raw)
    good = [(0, 29, 128), (3, 5, 1), (4, 6, 77), (4, 7, 127), (29 - 1, 8, 0), (1, 2, 13)]
    bad = [(0, 30, 5), (-1, 9, 5), (0, 10, 129), (0, 11, -1)]
    want = [a.view(torch.uint8).view(n_blocks, BLOCK, -1).clone() for a in arrays]
    for s, d, r in good:
        for w in want:
            w[d, :r] = w[s, :r]
    copies = torch.tensor(good + bad + [(12, 13, 128)], dtype=torch.int32, device="cuda")
    status = torch.tensor([len(good + bad), 0, 0, 0], dtype=torch.int32, device="cuda")
    mla.mla_blocks_copy(layer.config(mla), cache.struct, copies, status)
    torch.cuda.synchronize()
    assert status.tolist() == [len(good + bad), mla.MLA_DEVERR_BLOCK, 0, 0]
    for a, w in zip(arrays, want):
        assert torch.equal(a.view(torch.uint8).view(n_blocks, BLOCK, -1), w)


def test_copy_behind_32_bit_offsets():
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import LatentCache
    layer = Layer(d_c=256, seed=2)
    cache = LatentCache(layer.config(mla), 1, 128, "cuda", block_table=np.zeros((1, 1), dtype=np.int32), n_blocks=70000)
    assert cache.c_kv.numel() * 2 > 2 ** 32
    row = torch.randn(256).to(torch.bfloat16).cuda()
    cache.c_kv[69999, 5] = row
    copies = torch.tensor([(69999, 68000, 6)], dtype=torch.int32, device="cuda")
    status = torch.tensor([1, 0, 0, 0], dtype=torch.int32, device="cuda")
    mla.mla_blocks_copy(layer.config(mla), cache.struct, copies, status)
    assert torch.equal(cache.c_kv[68000, 5], row) and not cache.c_kv[68000, 6:].any() and status[1] == 0


def test_ring_copy():
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import LatentCache
    layer = Layer(d_c=96, cache="int4_r128", seed=3)
    cache = LatentCache(layer.config(mla), 5, 256, "cuda")
    cache.c_resid.copy_(torch.randn_like(cache.c_resid))
    cache.resid_pos.copy_(torch.randint(-1, 300, cache.resid_pos.shape, device="cuda"))
    ring, pos = cache.c_resid.clone(), cache.resid_pos.clone()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mla.mla_ring_copy(layer.config(mla), cache.struct, i(0, 0, 4, 2, 3), i(1, 2, 4, 9, 1), status)
    torch.cuda.synchronize()
    # (2, 9) is out of range, (3, 1) the second pair for row 1
    for d in (1, 2):
        ring[d], pos[d] = ring[0], pos[0]
    assert torch.equal(cache.c_resid, ring) and torch.equal(cache.resid_pos, pos)
    assert status[1] == mla.MLA_DEVERR_ROW


def test_fork_leaves_skipped_rings():
    """A pair that the fork skips for its source's length keeps its ring as well."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=96, cache="int4_r128", seed=3)
    pool = BlockPool(4, 256, 8)
    cache = pool.layer(layer.config(mla))
    cache.c_resid.copy_(torch.randn_like(cache.c_resid))
    ring, table = cache.c_resid.clone(), pool.table.clone()
    pool.fork([0, 2], [1, 3], [257, 0, 100, 0])
    torch.cuda.synchronize()
    ring[3] = ring[2]
    assert torch.equal(cache.c_resid, ring) and torch.equal(pool.table, table)
    assert pool.errors() == mla.MLA_DEVERR_SEQ_LEN


def test_pool_calls_on_another_stream():
    """Arguments that a call has to convert are converted on the call's stream, not on a busy one."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=64, seed=3)
    pool = BlockPool(4, 1024, 32)
    cache = pool.layer(layer.config(mla))
    i64 = lambda *x: torch.tensor(x, device="cuda")  # noqa: E731
    zero, lens, more, src, dst = i64(0, 0, 0, 0), i64(300, 0, 130, 0), i64(301, 301, 131, 131), i64(0, 2), i64(1, 3)
    forked = i64(300, 300, 130, 130)
    cache.c_kv.normal_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)   # the current stream is busy from here on
    for stream, call in [(side, lambda s: pool.reserve(zero, lens, stream=s)), (side, lambda s: pool.fork(src, dst, lens, stream=s)),
                         (side.cuda_stream, lambda s: pool.reserve(forked, more, stream=s)),
                         (side.cuda_stream, lambda s: pool.trim(more, 0, 150, stream=s)), (side, lambda s: pool.compact(stream=s))]:
        call(stream)
    side.synchronize()
    with torch.cuda.stream(side):
        assert pool.errors() == 0
        # rows [0 1 5] [0 1 2] [3 6] [3 4] with 2 and 4 copied on write; block 0 hidden by the window, 6 moved there
        assert pool.table[:, :3].tolist() == [[-1, 1, 5], [-1, 1, 2], [3, 0, -1], [3, 4, -1]] and pool.in_use() == 6
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", [dict(d_c=64), dict(d_c=128, cache="int4_r128")], ids=["bf16", "int4_r128"])
def test_serving_run(kind):
    """Two prompts, three samples of each by forking, steps with room made, appended, attended
    with a window, trimmed and compacted on the way: every step's output equals the definition
    over the sample's own tokens, and at the end every block is accounted for and freed."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(**kind, seed=4)
    n_sink, window, B, T_cap, n_blocks = 3, 150, 6, 1024, 40
    prompts, steps = [200, 333], 60
    pool = BlockPool(B, T_cap, n_blocks)
    cache = pool.layer(layer.config(mla))
    plan = layer.plan(mla)
    lens = np.zeros(B, dtype=np.int32)
    seqs = [layer.sequence(prompts[b % 2] + steps) for b in range(2)] * 3
    own = [layer.sequence(prompts[b % 2] + steps) for b in range(B)]
    for b in range(B):   # sample b: the prompt of b % 2, then its own tokens
        P = prompts[b % 2]
        s = {k: (torch.cat([seqs[b][k][:P], own[b][k][P:]]) if k not in ("L", "ring") else own[b][k]) for k in own[b]}
        if cache.c_resid is not None:   # the stored int4 values; the ring holds its own below
            full = layer.sequence(P + steps)
            s["int4"] = _int4_values(layer, s)
            s["exact"] = torch.cat([_exact_rows(layer, seqs[b % 2], P), _exact_rows(layer, own[b], P + steps)[P:]]) \
                if full else None
        own[b] = s

    def write(b, t0, t1):   # rows as an append would store them
        s = own[b]
        cache.set_latent_rows(b, t0, s["c_kv"][t0:t1])
        cache.set_k_rope_tokens(b, t0, s["kr"][t0:t1])
        if cache.c_scales is not None:
            cache.set_scale_rows(b, t0, s["c_scales"][t0:t1])
        if cache.c_resid is not None:
            t = torch.arange(max(t0, t1 - 128), t1)
            cache.c_resid[b, t % 128] = s["exact"][t].to(cache.c_resid)
            cache.resid_pos[b, t % 128] = t.to(cache.resid_pos)

    new = lens.copy()
    new[:2] = prompts
    pool.reserve(lens, new)
    lens = new
    for b in (0, 1):
        write(b, 0, prompts[b])
    pool.fork([0, 0, 1, 1], [2, 4, 3, 5], lens)
    lens = np.array([prompts[b % 2] for b in range(B)], dtype=np.int32)
    assert pool.in_use() == 2 + 3
    ws = torch.empty(mla.mla_decode_workspace_bytes(plan, B), dtype=torch.uint8, device="cuda")
    for step in range(steps):
        pool.reserve(lens, lens + 1)
        lens = lens + 1
        for b in range(B):
            write(b, int(lens[b]) - 1, int(lens[b]))
        if step % 7 == 3:
            pool.trim(lens, n_sink, window)
        if step % 11 == 5:
            pool.compact()
            assert pool.in_use() == 0 or int(torch.nonzero(pool.refs).max()) == pool.in_use() - 1
        q = layer.queries(B)
        out = torch.empty_like(q, device="cuda")
        mla.mla_decode_window(plan, cache.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), q.cuda(), out,
                              ws, n_sink, window)
        assert mla.mla_device_error(plan) == 0 and pool.errors() == 0
        if step in (0, 1, 30, steps - 1):
            for b in range(B):
                seq = {"c": _latent(own[b], int(lens[b])), "kr": own[b]["kr"][:int(lens[b])]}
                ref = layer.reference(q[b], seq, int(lens[b]) - 1, n_sink, window).numpy()
                assert_close(out[b].double().cpu().numpy(), ref, "bf16", f"step {step} sample {b}")
    named = pool.table[pool.table >= 0].long()
    assert torch.equal(torch.bincount(named.cpu(), minlength=n_blocks).int(), pool.refs.cpu())
    pool.trim(np.zeros(B), 0, 0)
    assert pool.in_use() == 0 and bool((pool.table == -1).all()) and pool.errors() == 0
    plan.close()


def _int4_values(layer, s):
    codes = s["c_kv"].int()
    v = torch.stack([codes & 15, codes >> 4], -1).reshape(len(codes), -1)
    return (v - 16 * (v >= 8)).double() * s["c_scales"].double().repeat_interleave(32, 1)


def _exact_rows(layer, s, L):
    """Unquantised rows near the stored ones (a ring row need not equal its int4 row)."""
    g = torch.Generator().manual_seed(int(s["c_kv"][:4].long().sum()))
    return (_int4_values(layer, s)[:L] + 0.1 * torch.randn(L, layer.d_c, generator=g)).to(layer.td)


def _latent(s, L):
    if "exact" not in s:
        return s["c"][:L]
    c = s["int4"][:L].clone()
    c[max(0, L - 128):] = s["exact"][max(0, L - 128):L].double()
    return c


def test_pool_calls_in_a_graph():
    """A step's bookkeeping captured once and replayed while the lengths move on."""
    import mha_mla_latent_b200 as mla
    B, C, n_blocks = 4, 6, 40
    table = np.full((B, C), -1, dtype=np.int32)
    table[:, 0] = [7, 7, 8, 9]
    refs = np.bincount(table[table >= 0], minlength=n_blocks).astype(np.int32)
    lens = np.array([100, 100, 120, 127], dtype=np.int32)
    d = Dev(table, refs)
    cur, nxt = d.up(lens), d.up(lens + 50)
    args = (d.table, d.refs, cur, nxt, d.table, d.refs, d.copies, d.status, d.ws)
    trim = (d.table, d.refs, nxt, 1, 130, d.table, d.refs, d.status)
    warm = Dev(table, refs)
    mla.mla_blocks_reserve(warm.table, warm.refs, cur, nxt, warm.table, warm.refs, warm.copies, warm.status, warm.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_blocks_reserve(*args)
        mla.mla_blocks_trim(*trim)
        cur.copy_(nxt)
        nxt.add_(50)
    for _ in range(8):
        graph.replay()
        want = m_reserve(table, refs, lens, lens + 50)
        table, refs = m_trim(want[0], want[1], lens + 50, 1, 130)
        lens = lens + 50
        torch.cuda.synchronize()
        assert np.array_equal(d.table.cpu().numpy(), table) and np.array_equal(d.refs.cpu().numpy(), refs)
        assert d.status[1] == 0


@pytest.mark.parametrize("n", [400, 300])   # with and without ring rows of the prefix left
def test_ring_of_a_cut_fork(n):
    """A fork of a shorter prefix than the source's own length takes no ring row of the tokens behind
    it: what the sequence appends there itself is in the window at full precision, as if the source
    had never been longer.  Cutting a row to its own length does the same."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=96, cache="int4_r128", seed=5)
    cfg = layer.config(mla)
    g = torch.Generator().manual_seed(1)
    W = [(torch.randn(64, n, generator=g) * 64 ** -0.5).to(layer.td) for n in (layer.d_c, layer.n_kv * layer.d_h)]
    plan = mla.mla_plan_create(cfg, *W, torch.from_numpy(layer.pairs), layer.W_uk, layer.W_uv)
    cut, more = 250, 40
    x = torch.randn(n, 64, generator=g).to(layer.td).cuda()
    y = torch.randn(more, 64, generator=g).to(layer.td).cuda()
    pool = BlockPool(3, 512, 20)
    cache = pool.layer(cfg)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def append(b, t0, rows):
        k = rows.shape[0]
        mla.mla_append(plan, rows, i32([b] * k), i32(range(t0, t0 + k)), cache.struct)

    pool.reserve([0, 0, 0], [n, 0, 0])
    append(0, 0, x)
    pool.fork([0, 0], [1, 0], [cut, 0, 0])
    assert int(cache.resid_pos[:2].max()) < cut
    kept = torch.arange(min(n - 128, cut), cut)           # ring rows of the prefix that were not written over
    for b in (0, 1):
        assert cache.resid_pos[b, kept.cuda() % 128].tolist() == kept.tolist()
    pool.reserve([cut, cut, 0], [cut + more, cut + more, cut + more])
    for b in (0, 1):
        append(b, cut, y)
    append(2, cut, y)                           # a ring that never held anything else
    t = torch.arange(cut, cut + more).cuda()
    torch.cuda.synchronize()
    for b in (0, 1):
        assert cache.resid_pos[b, t % 128].tolist() == t.tolist()
        assert torch.equal(cache.c_resid[b, t % 128], cache.c_resid[2, t % 128])
    assert pool.errors() == 0 and mla.mla_device_error(plan) == 0
    plan.close()


def m_reserve_shared(table, refs, lens, new):
    """m_reserve where columns behind the length may hold blocks: those that others hold too are
    given up for new ones."""
    B, C = table.shape
    out, cnt, copies, err = table.copy(), refs.copy(), [], 0
    free = [i for i in range(len(refs)) if refs[i] <= 0]
    writers = {}
    for b in range(B):
        L, N = int(lens[b]), int(new[b])
        if L % BLOCK and N > L and table[b][L // BLOCK] >= 0:
            writers.setdefault(int(table[b][L // BLOCK]), []).append(b)
    n0 = len(free)
    for b in range(B):
        L, N = int(lens[b]), int(new[b])
        if L % BLOCK and N > L:
            e = int(table[b][L // BLOCK])
            if refs[e] > 1 and (refs[e] > len(writers[e]) or writers[e][-1] != b):
                cnt[e] -= 1
                out[b][L // BLOCK] = free.pop(0)
                copies.append((e, int(out[b][L // BLOCK]), L % BLOCK))
                cnt[out[b][L // BLOCK]] += 1
        for j in range(blocks_of(L), blocks_of(N)):
            e = int(table[b][j])
            if e >= 0 and refs[e] <= 1:
                continue
            if e >= 0:
                cnt[e] -= 1
            out[b][j] = free.pop(0)
            cnt[out[b][j]] += 1
    return out, cnt, copies, err, n0 - len(free)


@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("size", [(2, 6, 40), (5, 12, 200), (40, 60, 6000), (1200, 5, 20000)], ids=str)
def test_reserve_behind_a_rolled_back_length(size, inplace):
    """Sequences that went back to a shorter length (drafted tokens that were not taken) still name
    the blocks behind it, which forks may share: a reserve gives them blocks of their own there."""
    B, C, n_blocks = size
    rng = np.random.default_rng(B)
    for trial in range(3):
        table, refs, lens = random_state(rng, B, C, n_blocks, share=0.8, holes=0.1 * (trial == 1))
        back = np.where(rng.random(B) < 0.8, (lens * rng.random(B)).astype(np.int64), lens)
        back = np.where(rng.random(B) < 0.2, back // BLOCK * BLOCK, back)
        for b in range(B):   # a partly filled last block has to be there
            if back[b] % BLOCK and table[b][back[b] // BLOCK] < 0:
                back[b] = back[b] // BLOCK * BLOCK
        new = np.minimum(back + rng.choice([0, 1, 129, 700, 9000], size=B), C * BLOCK)
        d = Dev(table, refs)
        want = m_reserve_shared(table, refs, back, new)
        got = d.call("reserve", d.up(back), d.up(new), inplace=inplace)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert got[2].tolist() == [len(want[2]), 0, int((want[1] > 0).sum()), want[4]]
        assert d.listed(len(want[2])) == want[2]
        # what a sequence may write into is its own
        held = np.bincount(got[0][got[0] >= 0], minlength=n_blocks)
        assert (got[1] == held).all()
        for b in np.nonzero(new > back)[0]:
            assert (held[got[0][b, int(back[b]) // BLOCK:blocks_of(int(new[b]))]] == 1).all()


def test_a_rolled_back_sample_leaves_the_others_alone():
    """Two samples share everything, one goes back and writes other tokens: the other's rows stay."""
    import mha_mla_latent_b200 as mla
    from mha_mla_latent_b200.cache import BlockPool
    layer = Layer(d_c=64, seed=6)
    pool = BlockPool(2, 1024, 20)
    cache = pool.layer(layer.config(mla))
    seq, other = layer.sequence(600), layer.sequence(600)
    pool.reserve([0, 0], [600, 0])
    cache.set_latent_rows(0, 0, seq["c_kv"])
    pool.fork([0], [1], [600, 0])
    for at in (300, 256):
        pool.reserve([at, 600], [580, 600])
        cache.set_latent_rows(0, at, other["c_kv"][at:580])
        assert torch.equal(cache.latent_rows(1, 0, 600).cpu(), seq["c_kv"])
        assert torch.equal(cache.latent_rows(0, 0, 580).cpu(), torch.cat([seq["c_kv"][:at], other["c_kv"][at:580]]))
        pool.fork([1], [0], [0, 600])
    assert pool.errors() == 0
