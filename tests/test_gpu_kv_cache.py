"""The paged 8-bit cache: rotary table, rotated append, reading back and
attention over it, against plain implementations (tests/kv_reference.py)."""
import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from w8a8_post_quantization_calibrate_b200 import sq  # noqa: E402

DEV = torch.device("cuda", 0)


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


def cu_of(lens):
    return np.concatenate(([0], np.cumsum(lens))).astype(np.int64).tolist()


class Pages:
    """A cache on both sides, random codes in it, pages in random order."""

    def __init__(self, lens, heads, d, ps, sb, seed, spare=2, garbage_scales=False):
        rng = np.random.default_rng(seed)
        need = [-(-max(n, 0) // ps) for n in lens]
        self.n = sum(need) + spare
        order = rng.permutation(self.n)
        self.most = max(max(need), 1)
        self.table = np.full((len(lens), self.most), 2 ** 30, np.int64)   # entries behind the last token: never read
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.k, self.v = (rng.integers(-127, 128, (self.n, heads, ps, d)).astype(np.int8) for _ in range(2))
        shape = (self.n, heads, ps // sb)
        self.ks, self.vs = (rng.uniform(0.005, 0.03, shape).astype(np.float32) for _ in range(2))
        if garbage_scales:   # blocks that hold no token: scales that must not matter
            used = np.zeros((self.n, ps // sb), bool)
            for b, n in enumerate(lens):
                for s0 in range(0, n, sb):
                    used[self.table[b, s0 // ps], s0 % ps // sb] = True
            for s in (self.ks, self.vs):
                s[~np.broadcast_to(used[:, None], shape)] = np.nan
        self.cache = sq.KvCache(*(torch.from_numpy(x.copy()).to(DEV) for x in (self.k, self.v, self.ks, self.vs)))
        self.dev_table = torch.from_numpy(self.table.astype(np.int32)).to(DEV)

    def check_equal(self, what):
        torch.cuda.synchronize()
        for name, mine, theirs in zip(("k", "v", "k_scale", "v_scale"), (self.k, self.v, self.ks, self.vs), self.cache):
            got = theirs.cpu().numpy()
            if got.dtype == np.float32:
                got, mine = got.view(np.uint32), mine.view(np.uint32)
            bad = np.argwhere(got != mine)
            assert bad.size == 0, f"{what} {name}: {len(bad)} differ, first {bad[:3].tolist()}: " \
                f"{got[tuple(bad[0])]} for {mine[tuple(bad[0])]}"


# ------------------------------------------------------------------ table
@pytest.mark.parametrize("first,n,rot,theta,scaling", [
    (0, 1, 16, 1e4, {}), (0, 100, 128, 1e4, {}), (5, 33, 64, 5e5, dict(factor=4.0)),
    (1_000_000, 70, 128, 1e6, dict(factor=8.0, low_turns=1.0, high_turns=4.0, original_len=8192, magnitude=1.2)),
    (2 ** 31 - 40, 40, 32, 1e4, {}), (0, 257, 256, 1e4, dict(magnitude=0.5))])
def test_rope_table(first, n, rot, theta, scaling):
    got = sq.sq_rope_table(n, rot, theta, first_pos=first, **scaling).cpu().numpy()
    kw = {"factor": "factor", "low_turns": "low", "high_turns": "high", "original_len": "orig", "magnitude": "mag"}
    want = ref.rope_table(first, n, rot, theta, **{kw[k]: v for k, v in scaling.items()})
    # one rounding to fp32, and the angle's fp64 error: a few 2^-53 of its size on both sides
    bound = 2.0 ** -24 * np.abs(want) + scaling.get("magnitude", 1.0) * (first + n) * 2.0 ** -48 + 1e-13
    assert np.all(np.abs(got - want) <= bound), np.abs(got - want).max()


# ------------------------------------------------------------------ append
APPENDS = [
    # new lens, ctx, hq, h, d, rot, ps, sb, pairs, dtype
    ([1], [0], 4, 1, 128, 128, 16, 16, False, torch.bfloat16),
    ([1, 1, 1, 1], [5, 16, 63, 64], 8, 2, 128, 128, 64, 16, False, torch.bfloat16),
    ([1, 0, 3], [31, 7, 0], 2, 2, 64, 32, 32, 1, True, torch.float32),
    ([37, 1, 130, 0, 16], [3, 100, 0, 9, 48], 12, 4, 128, 64, 64, 64, True, torch.bfloat16),
    ([50, 20], [13, 127], 3, 3, 64, 64, 128, 128, False, torch.float32),
    ([200], [60], 9, 1, 128, 16, 128, 128, False, torch.bfloat16),
    ([19, 40], [14, 2], 0, 5, 64, 0, 16, 4, False, torch.bfloat16),
    ([100, 33], [40, 11], 40, 8, 128, 96, 32, 32, True, torch.float32),
    ([17] * 40, [(7 * i) % 50 for i in range(40)], 4, 2, 64, 64, 16, 2, False, torch.bfloat16),
]


def _inputs(t, hq, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((t, hq + 2 * h, d), generator=g)
    qkv[:, :, :3] *= 9.0
    qkv = qkv.to(dtype)
    return qkv, qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_matches_the_formula_bit_for_bit(case):
    new, ctx, hq, h, d, rot, ps, sb, pairs, dtype = APPENDS[case]
    pg = Pages([a + b for a, b in zip(new, ctx)], h, d, ps, sb, seed=case)
    cu, t = cu_of(new), sum(new)
    pad = 3   # rows behind the last sequence
    qkv, q, k, v = _inputs(t + pad, hq, h, d, dtype, seed=case)
    table = ref.rope_table(0, max(a + b for a, b in zip(new, ctx)), max(rot, 2), 1e4).astype(np.float32)
    dq = qkv.to(DEV)
    q_out = torch.full((t + pad, hq, d), 7.0, dtype=dtype, device=DEV)
    k_out = torch.full((t + pad, h, d), 7.0, dtype=dtype, device=DEV)
    sq.sq_rope_kv_append(dq[:, :hq] if hq else None, dq[:, hq:hq + h], dq[:, hq + h:], pg.cache, pg.dev_table, ints(ctx),
                         ints(cu), table=torch.from_numpy(table).to(DEV) if rot else None, interleaved=pairs,
                         q_out=q_out if hq else None, k_out=k_out)
    assert sq.sq_get_status() == sq.SQ_OK
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(new, ctx)])
    f = [x[:t].float().numpy() for x in (q, k, v)]
    if rot:
        f[0], f[1] = ref.rotate(f[0], table[pos], pairs), ref.rotate(f[1], table[pos], pairs)
    ref.append(pg.k, pg.ks, f[1], pg.table, ctx, cu)
    ref.append(pg.v, pg.vs, f[2], pg.table, ctx, cu)
    pg.check_equal("append")
    for name, got, want in (("q", q_out, f[0]), ("k", k_out, f[1])):
        got = got.float().cpu().numpy()
        assert np.array_equal(got[:t], ref.rounded(want, dtype)), name
        assert np.all(got[t:] == 7.0), f"{name}: rows behind the last sequence were written"


def test_append_token_by_token_requantizes_within_its_bound():
    """One block filled token by token: its scale only grows, and each growth
    moves what is held by at most half a step of the new scale."""
    h, d, ps, sb = 2, 128, 32, 32
    pg = Pages([32], h, d, ps, sb, seed=3)
    g = torch.Generator().manual_seed(5)
    x = torch.randn((32, 2 * h, d), generator=g) * torch.linspace(0.5, 3.0, 32)[:, None, None]
    xd = x.to(DEV)
    moved = np.zeros(h)
    last = np.zeros(h)
    for i in range(32):
        sq.sq_rope_kv_append(None, xd[i:i + 1, :h], xd[i:i + 1, h:], pg.cache, pg.dev_table, ints([i]), ints([0, 1]))
        scale = pg.cache.k_scale.cpu().numpy()[pg.table[0, 0], :, 0].astype(np.float64)
        assert np.all(scale >= last)
        moved += np.where(scale > last, 0.5 * scale, 0.0)
        moved = np.where(scale > last, moved, np.maximum(moved, 0.5 * scale))
        last = scale
        got, _ = sq.sq_kv_read(pg.cache, pg.dev_table, ints([0]), ints([0, i + 1]), i + 1, dtype=torch.float32)
        err = np.abs(got.cpu().numpy().astype(np.float64) - x[:i + 1, :h].numpy()).max((0, 2))
        assert np.all(err <= moved * (1 + 2.0 ** -20) + last * 127 * 2.0 ** -22)
    assert sq.sq_get_status() == sq.SQ_OK


def test_append_zero_blocks_and_growth_from_zero():
    pg = Pages([20], 1, 64, 32, 32, seed=9)
    x = torch.zeros((10, 2, 64), device=DEV)
    sq.sq_rope_kv_append(None, x[:, :1], x[:, 1:], pg.cache, pg.dev_table, ints([0]), ints([0, 10]))
    p = pg.table[0, 0]
    assert float(pg.cache.k_scale[p, 0, 0]) == 0.0 and int(pg.cache.k[p, 0, :10].abs().sum()) == 0
    y = torch.full((1, 2, 64), 2.54, device=DEV)
    sq.sq_rope_kv_append(None, y[:, :1], y[:, 1:], pg.cache, pg.dev_table, ints([10]), ints([0, 1]))
    assert torch.all(pg.cache.k[p, 0, 10] == 127) and int(pg.cache.k[p, 0, :10].abs().sum()) == 0
    assert float(pg.cache.v_scale[p, 0, 0]) == float(np.float32(2.54) / np.float32(127))
    assert sq.sq_get_status() == sq.SQ_OK


def test_append_in_place():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((20, h, 128), generator=g).to(DEV) for h in (4, 2, 2))
    table = sq.sq_rope_table(64, 128)
    args = (ints([7, 0]), ints([0, 12, 20]))
    a, b = Pages([19, 8], 2, 128, 16, 8, seed=4), Pages([19, 8], 2, 128, 16, 8, seed=4)
    qo, ko = sq.sq_rope_kv_append(q, k, v, a.cache, a.dev_table, *args, table=table, want_k=True)
    q2, k2 = q.clone(), k.clone()
    sq.sq_rope_kv_append(q2, k2, v, b.cache, b.dev_table, *args, table=table, q_out=q2, k_out=k2)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    for x, y in zip(a.cache, b.cache):
        assert torch.equal(x, y)


def test_append_bad_pages_and_positions_are_skipped_and_reported():
    h, d, ps, sb = 2, 64, 16, 16
    new, ctx = [20, 5, 6], [0, 30, 2]
    pg = Pages([20, 35, 8], h, d, ps, sb, seed=6)
    pg.table[0, 1] = pg.n + 5      # behind the cache
    pg.table[2, 0] = -1
    pg.dev_table = torch.from_numpy(pg.table.astype(np.int32)).to(DEV)
    t = sum(new)
    qkv, q, k, v = _inputs(t, 2, h, d, torch.float32, seed=2)
    dq = qkv.to(DEV)
    rows = 33    # the table ends inside sequence 1
    table = ref.rope_table(0, rows, d, 1e4).astype(np.float32)
    qo, ko = sq.sq_rope_kv_append(dq[:, :2], dq[:, 2:2 + h], dq[:, 2 + h:], pg.cache, pg.dev_table, ints(ctx), ints(cu_of(new)),
                                  table=torch.from_numpy(table).to(DEV), want_k=True)
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS
    assert sq.sq_get_status() == sq.SQ_OK
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(new, ctx)])
    inside = pos < rows
    cs = table[np.minimum(pos, rows - 1)]
    kr = ref.rotate(k.numpy(), cs, False)
    ref.append(pg.k, pg.ks, kr, pg.table, ctx, cu_of(new), limit=rows)
    ref.append(pg.v, pg.vs, v.numpy(), pg.table, ctx, cu_of(new), limit=rows)
    pg.check_equal("append with bad pages")
    got = ko.cpu().numpy()
    assert np.array_equal(got[inside], kr[inside]) and np.isnan(got[~inside]).all()
    assert np.isnan(qo.cpu().numpy()[~inside]).all() and not np.isnan(qo.cpu().numpy()[inside]).any()


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("d,ps,sb,h,dtype", [(64, 16, 1, 3, torch.float32), (128, 64, 16, 8, torch.bfloat16),
                                             (128, 128, 128, 1, torch.float32), (64, 32, 8, 40, torch.bfloat16)])
def test_read(d, ps, sb, h, dtype):
    lens, first = [1, 0, 77, 130, 16], [0, 0, 5, 129, 3]
    pg = Pages(lens, h, d, ps, sb, seed=d + ps)
    n = [max(0, a - b) for a, b in zip(lens, first)]
    t = sum(n)
    k = torch.full((t + 2, h, d), 5.0, dtype=dtype, device=DEV)
    v = torch.full((t + 2, h, d), 5.0, dtype=dtype, device=DEV)
    sq.sq_kv_read(pg.cache, pg.dev_table, ints(first), ints(cu_of(n)), t + 2, k_out=k, v_out=v)
    assert sq.sq_get_status() == sq.SQ_OK
    for got, codes, scales in ((k, pg.k, pg.ks), (v, pg.v, pg.vs)):
        want = np.concatenate([ref.held(codes, scales, pg.table[b], first[b], first[b] + n[b]) for b in range(len(n))])
        got = got.float().cpu().numpy()
        assert np.array_equal(got[:t], ref.rounded(want, dtype)) and np.all(got[t:] == 5.0)


def test_read_bad_pages_give_nan():
    pg = Pages([40], 2, 64, 16, 16, seed=8)
    pg.dev_table[0, 1] = pg.n
    k, v = sq.sq_kv_read(pg.cache, pg.dev_table, ints([0]), ints([0, 50]), 50, dtype=torch.float32)   # 48 tokens fit the table
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS
    for x in (k, v):
        bad = torch.isnan(x).flatten(1).all(1).cpu().numpy()
        assert np.array_equal(np.nonzero(bad)[0], list(range(16, 32)) + [48, 49])
        assert torch.isnan(x).flatten(1).any(1).cpu().numpy().sum() == 18


# ------------------------------------------------------------------ attention
ATTENTIONS = [
    # lens, q_len, hq, h, d, ps, sb, dtype
    ([1], 1, 4, 1, 128, 16, 16, torch.bfloat16),
    ([0, 1, 15, 16, 17, 63, 64, 65], 1, 8, 2, 128, 16, 1, torch.bfloat16),
    ([700, 3, 0, 129], 1, 32, 8, 128, 64, 16, torch.bfloat16),
    ([5, 300, 2, 0], 4, 8, 8, 128, 32, 8, torch.float32),
    ([260, 77], 1, 4, 4, 64, 128, 128, torch.float32),
    ([33, 1000], 2, 16, 1, 64, 64, 4, torch.bfloat16),
    ([400, 9], 16, 16, 2, 128, 16, 16, torch.bfloat16),
    ([50] * 70, 3, 12, 4, 64, 32, 32, torch.bfloat16),
    ([5000], 1, 8, 1, 128, 128, 64, torch.bfloat16),
    ([2100, 1], 5, 25, 5, 128, 64, 2, torch.float32),
    ([1500, 1500, 1500], 1, 64, 8, 128, 64, 64, torch.float32),
    ([129] * 3, 7, 17, 1, 128, 16, 16, torch.bfloat16),
]


def check_attention(pg, lens, q, out, lse, scale, dtype, what=""):
    n, l, hq, d = q.shape
    h = pg.k.shape[1]
    g = hq // h
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    qn = q.float().cpu().numpy()
    f32 = dtype == torch.float32
    for b in range(n):
        k, v = (ref.held(c, s, pg.table[b], 0, lens[b]) for c, s in ((pg.k, pg.ks), (pg.v, pg.vs)))
        seen = np.arange(lens[b])[None] <= (lens[b] - l + np.repeat(np.arange(l), g))[:, None]
        for j in range(h):
            rows = qn[b, :, j * g:(j + 1) * g].reshape(l * g, d)
            want, wlse, bound, lbound = ref.attention(rows, k[:, j], v[:, j], scale, seen, 2.0 ** -22 if f32 else 2.0 ** -11,
                                                      2.0 ** -24 if f32 else 2.0 ** -8, q_step=2.0 ** -24)
            got = out[b, :, j * g:(j + 1) * g].reshape(l * g, d)
            glse = lse[b, :, j * g:(j + 1) * g].reshape(l * g)
            assert np.all(np.abs(got - want) <= bound), \
                f"{what} seq {b} head {j}: {np.max(np.abs(got - want) / bound)} of the bound, rows {np.argwhere(np.abs(got - want) > bound)[:3].tolist()}"
            empty = ~seen.any(1) if lens[b] else np.ones(l * g, bool)
            assert np.all(got[empty] == 0.0) and np.all(np.isneginf(glse[empty]))
            assert np.all(np.abs(glse[~empty] - wlse[~empty]) <= lbound[~empty])


@pytest.mark.parametrize("case", range(len(ATTENTIONS)))
def test_attention(case):
    lens, l, hq, h, d, ps, sb, dtype = ATTENTIONS[case]
    pg = Pages(lens, h, d, ps, sb, seed=case, garbage_scales=True)
    g = torch.Generator().manual_seed(case)
    q = torch.randn((len(lens), l, hq, d), generator=g).to(dtype).to(DEV)
    out, lse = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints(lens), want_lse=True)
    assert sq.sq_get_status() == sq.SQ_OK
    check_attention(pg, lens, q, out, lse, d ** -0.5, dtype)
    again = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints(lens))
    assert torch.equal(out, again), "two calls differ"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,scale", [(1e4, 1e-5), (1e-30, 1e28), (3e37, 1e-38), (1.0, 2.0), (1.0, -0.05), (1.0, 0.0)])
def test_attention_scales_and_sizes_of_q(size, scale, dtype):
    """Queries of any fp32 size, scores from flat to one-hot."""
    lens, hq, h, d = [300, 40], 8, 2, 128
    pg = Pages(lens, h, d, 16, 16, seed=77)
    g = torch.Generator().manual_seed(3)
    q = (torch.randn((2, 1, hq, d), generator=g) * size).to(dtype).to(DEV)
    out, lse = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints(lens), scale=scale, want_lse=True)
    assert sq.sq_get_status() == sq.SQ_OK
    check_attention(pg, lens, q, out, lse, scale, dtype)


def test_attention_of_a_zero_query_is_the_mean():
    pg = Pages([100], 1, 128, 32, 4, seed=5)
    out, lse = sq.sq_kv_attention(torch.zeros((1, 1, 1, 128), device=DEV), pg.cache, pg.dev_table, ints([100]), want_lse=True)
    check_attention(pg, [100], torch.zeros((1, 1, 1, 128)), out, lse, 128 ** -0.5, torch.float32)


def test_attention_strided_queries_and_supplied_buffers():
    lens, hq, h, d = [90, 31, 64], 8, 4, 128
    pg = Pages(lens, h, d, 16, 16, seed=12)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((3 * 2, hq + 2 * h, d), generator=g).bfloat16().to(DEV)
    q = qkv.view(3, 2, hq + 2 * h, d)[:, :, :hq]
    out = torch.empty((3, 2, hq, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3, 2, hq), device=DEV)
    ws = torch.full((max(256, sq.sq_kv_attention_workspace_size(pg.cache, 3, 2, hq)),), 255, dtype=torch.uint8, device=DEV)
    o, s = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints(lens), out=out, lse=lse, workspace=ws)
    assert o is out and s is lse and sq.sq_get_status() == sq.SQ_OK
    check_attention(pg, lens, q, out, lse, d ** -0.5, torch.bfloat16)
    assert torch.equal(out, sq.sq_kv_attention(q.contiguous(), pg.cache, pg.dev_table, ints(lens)))


def test_attention_bad_pages_and_lengths_give_nan():
    lens = [40, 20, 33, 16]
    pg = Pages(lens, 2, 128, 16, 16, seed=13)
    pg.dev_table[0, 1] = pg.n        # behind the cache, inside the sequence
    pg.dev_table[2, 2] = -7
    q = torch.randn((4, 1, 4, 128), device=DEV)
    out, lse = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints([40, 20, 33, 1000]), want_lse=True)
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS and sq.sq_get_status() == sq.SQ_OK
    nan = torch.isnan(out).flatten(1)
    assert nan[0].all() and not nan[1].any() and nan[2].all() and nan[3].all()
    assert torch.isnan(lse[[0, 2, 3]]).all() and not torch.isnan(lse[1]).any()
    out = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints([16, 20, 32, -1]))   # the bad pages lie behind the tokens
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS
    nan = torch.isnan(out).flatten(1)
    assert not nan[:3].any() and nan[3].all()


def test_attention_on_another_stream_and_in_a_graph():
    """Captured once, replayed with new queries, lengths and codes; and a call
    on a side stream that the caller names."""
    lens, hq, h, d = [200, 1, 77], 16, 2, 128
    pg = Pages([400, 400, 400], h, d, 64, 16, seed=14)
    q, n = torch.randn((3, 1, hq, d), device=DEV).bfloat16(), ints(lens)
    out = torch.empty_like(q)
    ws = torch.empty(max(256, sq.sq_kv_attention_workspace_size(pg.cache, 3, 1, hq)), dtype=torch.uint8, device=DEV)
    want = [sq.sq_kv_attention(q, pg.cache, pg.dev_table, n)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.sq_kv_attention(q, pg.cache, pg.dev_table, n, out=out, workspace=ws)
    g.replay()
    assert torch.equal(out, want[0])
    q.copy_(torch.randn((3, 1, hq, d), device=DEV).bfloat16())
    n.copy_(ints([399, 0, 130]))
    pg.cache.k.neg_()
    want = sq.sq_kv_attention(q, pg.cache, pg.dev_table, n)
    g.replay()
    assert torch.equal(out, want) and not out[1].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sq.sq_kv_attention(q, pg.cache, pg.dev_table, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and sq.sq_get_status() == sq.SQ_OK


def test_offsets_beyond_32_bits():
    """A cache above 2^31 codes: the last pages are reached."""
    h, d, ps = 8, 128, 128
    pages = 2 ** 31 // (h * d * ps) + 40
    cache = sq.KvCache(torch.zeros((pages, h, ps, d), dtype=torch.int8, device=DEV),
                       torch.zeros((pages, h, ps, d), dtype=torch.int8, device=DEV),
                       torch.ones((pages, h, 1), device=DEV), torch.ones((pages, h, 1), device=DEV))
    table = ints([pages - 1, 0, pages - 2]).view(1, 3)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((300, 2 * h, d), generator=g).to(DEV)
    sq.sq_rope_kv_append(None, x[:, :h], x[:, h:], cache, table, ints([0]), ints([0, 300]))
    k, v = sq.sq_kv_read(cache, table, ints([0]), ints([0, 300]), 300, dtype=torch.float32)
    step = x.abs().amax() / 127
    assert (k - x[:, :h]).abs().max() <= step * 0.501 and (v - x[:, h:]).abs().max() <= step * 0.501
    q = torch.randn((1, 1, h, d), generator=g).to(DEV)
    out = sq.sq_kv_attention(q, cache, table, ints([300]))
    w = torch.softmax(torch.einsum("hd,thd->ht", q[0, 0].double(), k.double()) * d ** -0.5, -1)
    want = torch.einsum("ht,thd->hd", w, v.double())
    assert (out[0, 0].double() - want).abs().max() <= 1e-4 * v.abs().max()
    assert sq.sq_get_status() == sq.SQ_OK


@pytest.mark.parametrize("d,dtype,rows,tiles", [(128, torch.bfloat16, 1, 4), (128, torch.float32, 16, 4), (64, torch.bfloat16, 16, 8),
                                                (64, torch.float32, 1, 8), (128, torch.bfloat16, 8, 1), (128, torch.bfloat16, 2, 5)])
def test_attention_of_sequences_as_long_as_the_ring(d, dtype, rows, tiles):
    """Every fourth tile of 128 tokens (eighth for heads of 64) takes the place of an earlier one
    in shared memory; here it brings another sequence's queries there, and for every third
    sequence a bad page."""
    seqs, n, ps = 500, 128 * tiles, 64
    pg = Pages([n] * 2, 1, d, ps, 16, seed=tiles + d)
    table = pg.dev_table[torch.arange(seqs, device=DEV) % 2].contiguous()
    table[2::3, n // ps - 1] = pg.n
    g = torch.Generator().manual_seed(rows)
    q = torch.randn((seqs, 1, rows, d), generator=g).to(dtype).to(DEV)
    lens = ints([n] * seqs)
    out, lse = sq.sq_kv_attention(q, pg.cache, table, lens, want_lse=True)
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS and sq.sq_get_status() == sq.SQ_OK
    bad = torch.arange(seqs, device=DEV) % 3 == 2
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    for i in range(10):
        again = sq.sq_kv_attention(q, pg.cache, table, lens)
        assert torch.equal(again[~bad], out[~bad]), "two calls differ"
    for p in range(2):   # sequences on the same pages as rows of one product
        mine = torch.nonzero(~bad & (torch.arange(seqs, device=DEV) % 2 == p)).flatten()
        k, v = (ref.held(c, s, pg.table[p], 0, n)[:, 0] for c, s in ((pg.k, pg.ks), (pg.v, pg.vs)))
        qn = q[mine].float().cpu().numpy().reshape(-1, d)
        f32 = dtype == torch.float32
        want, wlse, bound, lbound = ref.attention(qn, k, v, d ** -0.5, np.ones((len(qn), n), bool), 2.0 ** -22 if f32 else 2.0 ** -11,
                                                  2.0 ** -24 if f32 else 2.0 ** -8, q_step=2.0 ** -24)
        assert np.all(np.abs(out[mine].float().cpu().numpy().reshape(-1, d) - want) <= bound)
        assert np.all(np.abs(lse[mine].cpu().numpy().reshape(-1) - wlse) <= lbound)
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS


def _value_scales(mode, vs, lens, table, ps, sb):
    """Value scales [pages, heads, blocks] of a test of zero and very unlike scales."""
    for b, n in enumerate(lens):
        for s0 in range(0, n, sb):
            at = (table[b, s0 // ps], slice(None), s0 % ps // sb)
            if mode == "all zero":
                vs[at] = 0.0
            elif mode == "first 32 zero":
                vs[at] *= s0 >= 32
            elif mode == "every other 32 zero":
                vs[at] *= s0 // 32 % 2
            elif mode == "first 640 zero":
                vs[at] *= s0 >= 640
            elif mode == "zero, tiny and ordinary":
                vs[at] *= (0.0, 2.0 ** -60, 1.0)[s0 // 16 % 3]
            elif mode == "2^-70 to 2^90":
                vs[at] *= 2.0 ** ((s0 // 16 * 37) % 161 - 70)
            elif mode == "near 1e30":
                vs[at] *= 2.0 ** 100


MODES = ["all zero", "first 32 zero", "every other 32 zero", "first 640 zero", "zero, tiny and ordinary", "2^-70 to 2^90", "near 1e30"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", MODES)
def test_attention_of_zero_and_very_unlike_value_scales(mode, dtype):
    """Blocks of zero values (scale 0, as the append writes them) anywhere, a lone token among them;
    sequences of one CTA and sequences that many share; codes that a scale of 0 makes 0."""
    lens, hq, h, d, ps, sb = [1, 20, 32, 33, 700, 5000], 6, 2, 128, 64, 16
    pg = Pages(lens, h, d, ps, sb, seed=21)
    _value_scales(mode, pg.vs, lens, pg.table, ps, sb)
    pg.cache.v_scale.copy_(torch.from_numpy(pg.vs))
    for l in (1, 5, 40):
        g = torch.Generator().manual_seed(l)
        q = torch.randn((len(lens), l, hq, d), generator=g).to(dtype).to(DEV)
        out, lse = sq.sq_kv_attention(q, pg.cache, pg.dev_table, ints(lens), want_lse=True)
        assert sq.sq_get_status() == sq.SQ_OK
        check_attention(pg, lens, q, out, lse, d ** -0.5, dtype, what=f"{mode}, {l} tokens,")
        if mode == "all zero":
            assert not out.any() and not torch.isnan(lse).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("steps", [40, 90, 200, 2000])
def test_attention_of_a_zero_value_with_a_score_far_above(steps, dtype):
    """Tokens of zero value whose scores are `steps` powers of two above all others, behind groups of
    ordinary ones in the same warp's share: the sum of the weights stays finite."""
    n, seqs, d, ps, sb = 1536, 300, 64, 64, 16
    pg = Pages([n], 1, d, ps, sb, seed=22)
    pg.k[:] = 0
    pg.ks[:] = 0.02
    high = np.arange(n) // sb % 40 == 30
    for p in np.nonzero(high)[0]:
        pg.k[pg.table[0, p // ps], 0, p % ps, 0] = 100
        pg.vs[pg.table[0, p // ps], 0, p % ps // sb] = 0.0
    for mine, theirs in zip((pg.k, pg.ks, pg.vs), (pg.cache.k, pg.cache.k_scale, pg.cache.v_scale)):
        theirs.copy_(torch.from_numpy(mine))
    q = torch.zeros((seqs, 1, 2, d), device=DEV)
    q[:, :, 0, 0] = 1.0      # head 1 is flat
    scale = steps * np.log(2.0) / (100 * 0.02)
    out, lse = sq.sq_kv_attention(q.to(dtype), pg.cache, pg.dev_table.expand(seqs, -1).contiguous(), ints([n] * seqs), scale=scale, want_lse=True)
    assert sq.sq_get_status() == sq.SQ_OK
    # the others have a score of 0 beside `high` of them at `steps` octaves
    v = ref.held(pg.v, pg.vs, pg.table[0], 0, n)[:, 0].astype(np.float64)
    for head, w in ((0, 2.0 ** -float(min(steps, 1000))), (1, 1.0)):
        p = np.where(high, 1.0, w)
        want = p @ v / p.sum()
        # fp16 weights (two parts for fp32) and their floor of 2^-25 of the reference's weight, sums over n, the output's rounding
        step, last = (2.0 ** -22, 2.0 ** -24) if dtype == torch.float32 else (2.0 ** -11, 2.0 ** -8)
        a = p @ np.abs(v) / p.sum()
        e = 2.0 ** -21 * (steps + 8) + 64 * 2.0 ** -23 * steps
        bound = 1.1 * ((step + 2 * e + n * 2.0 ** -23) * a + n * 2.0 ** -25 * w * np.abs(v).max() / p.sum() + last * np.abs(want)) + 1e-38
        got = out[:, 0, head].float().cpu().numpy()
        assert np.all(np.abs(got - want) <= bound), (head, np.max(np.abs(got - want) / bound))
        true = np.log(p.sum()) + (0.0 if head else steps * np.log(2.0))
        assert np.all(np.abs(lse[:, 0, head].cpu().numpy() - true) <= 1.1 * (e + n * 2.0 ** -23) + 2.0 ** -20 * abs(true) + 2.0 ** -22)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("steps", [12.3, 20.02, 25.02, 28.5])
def test_attention_of_many_small_weights_beside_a_large_one(steps, dtype):
    """One token of zero value weighs 2^steps times as much as each of 32,767 others, which are all of the
    result: a weight keeps 2^-32 of the largest, or fp16's relative 2^-11 (fp32: 2^-22)."""
    n, d, ps, sb = 32768, 64, 128, 128
    seqs = torch.cuda.get_device_properties(0).multi_processor_count   # a whole sequence for each CTA
    pg = Pages([n], 1, d, ps, sb, seed=23)
    pg.k[:] = 0
    pg.k[pg.table[0, 0], 0, 0, 0] = 100
    pg.v = np.abs(pg.v.astype(np.int16)).clip(60, 127).astype(np.int8)
    pg.v[pg.table[0, 0], 0, 0] = 0
    pg.ks[:], pg.vs[:] = 2.0 ** -6, 2.0 ** -5
    for mine, theirs in zip((pg.k, pg.v, pg.ks, pg.vs), pg.cache):
        theirs.copy_(torch.from_numpy(mine))
    q = torch.zeros((seqs, 1, 1, d), device=DEV, dtype=dtype)
    q[..., 0] = 1.0
    scale = float(np.float32(steps * np.log(2.0) / (100 * 2.0 ** -6)))
    out = sq.sq_kv_attention(q, pg.cache, pg.dev_table.expand(seqs, -1).contiguous(), ints([n] * seqs), scale=scale)
    assert sq.sq_get_status() == sq.SQ_OK
    v = ref.held(pg.v, pg.vs, pg.table[0], 0, n)[:, 0].astype(np.float64)
    p = np.full(n, np.exp(-scale * 100 * 2.0 ** -6))
    p[0] = 1.0
    want = p @ v / p.sum()
    step, last = (2.0 ** -22, 2.0 ** -24) if dtype == torch.float32 else (2.0 ** -11, 2.0 ** -8)
    e = 2.0 ** -21 * (steps + 16)      # the exponent's argument: scale, reference and difference in fp32
    bound = 1.1 * ((step + 2 * e + n * 2.0 ** -23) * want + n * 2.0 ** -32 * v.max() / p.sum() + last * want)
    err = np.abs(out[:, 0, 0].float().cpu().numpy() - want)
    assert np.all(err <= bound), np.max(err / bound)


def test_read_leaves_rows_before_the_first_sequence():
    """Rows that no sequence has, in front of the first and behind the last one, stay as they were."""
    pg = Pages([50, 20], 3, 64, 16, 4, seed=31)
    k, v = (torch.full((60, 3, 64), 5.0, device=DEV) for _ in range(2))
    sq.sq_kv_read(pg.cache, pg.dev_table, ints([17, 2]), ints([9, 30, 48]), 60, k_out=k, v_out=v)
    assert sq.sq_get_status() == sq.SQ_OK
    for got, codes, scales in ((k, pg.k, pg.ks), (v, pg.v, pg.vs)):
        got = got.cpu().numpy()
        want = np.concatenate([ref.held(codes, scales, pg.table[0], 17, 38), ref.held(codes, scales, pg.table[1], 2, 20)])
        assert np.array_equal(got[9:48], want) and np.all(got[:9] == 5.0) and np.all(got[48:] == 5.0)


def test_append_and_read_offsets_outside_the_rows_are_cut_and_reported():
    h, d, t = 2, 64, 100
    ctx = [5, 17]
    g = torch.Generator().manual_seed(8)
    x = torch.randn((t, 2 * h, d), generator=g).to(DEV)
    got = []
    for cu, status in (([0, 40, 100], sq.SQ_OK), ([0, 40, 150], sq.SQ_ERR_BOUNDS), ([0, 40, 2 ** 31 - 1], sq.SQ_ERR_BOUNDS)):
        pg = Pages([45 + 60, 17 + 60], h, d, 16, 8, seed=41)
        _, k = sq.sq_rope_kv_append(None, x[:, :h], x[:, h:], pg.cache, pg.dev_table, ints(ctx), ints(cu), want_k=True)
        assert sq.sq_get_status() == status and sq.sq_get_status() == sq.SQ_OK
        kr, vr = sq.sq_kv_read(pg.cache, pg.dev_table, ints(ctx), ints(cu), t, dtype=torch.float32)
        assert sq.sq_get_status() == status and sq.sq_get_status() == sq.SQ_OK
        got.append((k, kr, vr, *pg.cache))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    for cu in ([0, 60, 40], [-3, 40, 60], [0, 101, 60]):
        pg = Pages([200, 200], h, d, 16, 8, seed=42)
        sq.sq_rope_kv_append(None, x[:, :h], x[:, h:], pg.cache, pg.dev_table, ints(ctx), ints(cu))
        assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS
        sq.sq_kv_read(pg.cache, pg.dev_table, ints(ctx), ints(cu), t)
        assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS
