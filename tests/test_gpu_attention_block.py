"""The calls behind the QKV projection as they are used together: a layer's
attention block from the norm to the output projection's codes, for prompts and
for the tokens after them, against 64 bits; no call writes outside its
outputs; two calls at once."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from w8a8_post_quantization_calibrate_b200 import sq  # noqa: E402

DEV = torch.device("cuda", 0)
HQ, H, D, K = 8, 2, 128, 512
ROPE = dict(theta=5e5, factor=4.0, low_turns=1.0, high_turns=4.0, original_len=64)


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


class Block:
    """One layer's attention block over libsq: RMSNorm with the folded gain and
    int8 codes, W8A8 QKV projection, rotation and append, attention, codes for
    the output projection."""

    def __init__(self):
        g = torch.Generator().manual_seed(0)
        w = (torch.randn(((HQ + 2 * H) * D, K), generator=g) / K ** 0.5).bfloat16().to(DEV)
        self.s = torch.rand(K, generator=g).add_(0.5).to(DEV)
        self.gain = sq.sq_fold_norm_gain(torch.rand(K, generator=g).add_(0.5).to(DEV), self.s)
        self.wq, self.w_scale = sq.sq_fold_quant_weights(w, self.s)
        self.table = sq.sq_rope_table(256, D, **ROPE)
        self.ones = torch.ones(HQ * D, device=DEV)
        self.pages = ints([5, 0, 3, 1, 4, 2, 7, 6, 9, 8, 11, 10]).view(3, 4)
        self.cache = sq.KvCache.empty(12, H, D, page_size=32, scale_block=8)

    def qkv(self, x):
        xq, xs, _ = sq.sq_rmsnorm_quant_act(x, self.gain, 1e-5, want_inv_rms=False)
        y = sq.sq_w8a8_gemm(xq, xs, self.wq, self.w_scale, out_dtype=torch.bfloat16)
        y = y.view(x.shape[0], HQ + 2 * H, D)
        return y[:, :HQ], y[:, HQ:HQ + H], y[:, HQ + H:]

    def prompts(self, x, cu):
        q, k, v = self.qkv(x)
        q, k = sq.sq_rope_kv_append(q, k, v, self.cache, self.pages, ints([0, 0, 0]), cu, table=self.table, want_k=True)
        return (q, k, v), sq.sq_prompt_attention(q, k, v, cu)

    def step(self, x, ctx, cu):
        """One new token of every sequence; ctx [n] tokens before it."""
        q, k, v = self.qkv(x)
        q, _ = sq.sq_rope_kv_append(q, k, v, self.cache, self.pages, ctx, cu, table=self.table)
        return q, sq.sq_kv_attention(q.unsqueeze(1), self.cache, self.pages, ctx + 1)[:, 0]


def test_prompts_then_tokens():
    block = Block()
    lens = [40, 1, 90]
    cu = np.concatenate(([0], np.cumsum(lens))).tolist()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((sum(lens), K), generator=g).bfloat16().to(DEV)
    raw = [t.float().cpu().numpy() for t in block.qkv(x)]
    (q, k, v), out = block.prompts(x, ints(cu))
    codes = sq.sq_smooth_quant_act(out.reshape(-1, HQ * D), block.ones)
    assert sq.sq_get_status() == sq.SQ_OK
    # rotation by positions of its own sequence, table against its formula
    table = block.table.cpu().numpy()
    want = ref.rope_table(0, 256, D, 5e5, factor=4.0, low=1.0, high=4.0, orig=64)
    assert np.all(np.abs(table - want) <= 2.0 ** -24 * np.abs(want) + 1e-12)
    pos = np.concatenate([np.arange(n) for n in lens])
    for got, r in ((q, raw[0]), (k, raw[1])):
        assert np.array_equal(got.float().cpu().numpy(), ref.bf16(ref.rotate(r, table[pos], False)))
    o = out.float().cpu().numpy()
    for a, b in zip(cu, cu[1:]):
        n = b - a
        for j in range(HQ):
            t, _, bound, _ = ref.attention(q[a:b, j].float().cpu().numpy(), k[a:b, j // 4].float().cpu().numpy(), raw[2][a:b, j // 4],
                                           D ** -0.5, np.tril(np.ones((n, n), bool)), 2.0 ** -8, 2.0 ** -8)
            assert np.all(np.abs(o[a:b, j] - t) <= bound)
    scale = codes[1].cpu().numpy()
    amax = np.abs(o.reshape(sum(lens), -1)).max(1)
    assert np.array_equal(scale, (amax / np.float32(127)).astype(np.float32))

    # three more tokens of every sequence, the step captured once and replayed
    ctx, cu1 = ints(lens), ints([0, 1, 2, 3])
    xs = torch.randn((3, 3, K), generator=g).bfloat16().to(DEV)
    x_in = xs[0].clone()
    keep = [t.clone() for t in block.cache]
    block.step(x_in, ctx, cu1)                       # first launches outside of the capture
    for t, u in zip(block.cache, keep):
        t.copy_(u)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q1, o1 = block.step(x_in, ctx, cu1)
    for i in range(3):
        x_in.copy_(xs[i])
        graph.replay()
        assert sq.sq_get_status() == sq.SQ_OK
        for b, n in enumerate(lens):
            m = n + i + 1
            kk, vv = sq.sq_kv_read(block.cache, block.pages[b:b + 1], ints([0]), ints([0, m]), m, dtype=torch.float32)
            for j in range(HQ):
                t, _, bound, _ = ref.attention(q1[b, j:j + 1].float().cpu().numpy(), kk[:, j // 4].cpu().numpy(), vv[:, j // 4].cpu().numpy(),
                                               D ** -0.5, np.ones((1, m), bool), 2.0 ** -11, 2.0 ** -8, q_step=2.0 ** -24)
                assert np.all(np.abs(o1[b, j].float().cpu().numpy() - t[0]) <= bound[0])
            if i == 0:   # the prompt's keys as the cache holds them: half a step of their block's scale
                s = block.cache.k_scale[block.pages[b].long()].permute(0, 2, 1).reshape(-1, H).repeat_interleave(8, 0)[:n]
                err = (kk[:n] - torch.from_numpy(ref.rotate(raw[1][cu[b]:cu[b + 1]], table[:n], False)).to(DEV)).abs().amax(-1)
                # a block that was grown by the new token moved once more
                assert torch.all(err <= s * 1.0001)
        ctx += 1


@pytest.mark.parametrize("d,dtype,l", [(128, torch.bfloat16, 1), (64, torch.float32, 3)])
def test_no_call_writes_outside_its_outputs(d, dtype, l):
    lens, hq, h, ps = [70, 0, 33], 6, 2, 16
    g = torch.Generator().manual_seed(2)
    table = Guarded((80, d // 2, 2), torch.float32, DEV, seed=1)
    sq.sq_rope_table(80, d, table=table.t)
    table.check("rope_table")
    codes = [Guarded((8, h, ps, d), torch.int8, DEV, seed=2 + i) for i in range(2)]
    scales = [Guarded((8, h, ps // 4), torch.float32, DEV, seed=4 + i) for i in range(2)]
    cache = sq.KvCache(codes[0].t, codes[1].t, scales[0].t, scales[1].t)
    pages = ints([0, 1, 2, 3, 7, 0, 0, 0, 0, 0, 4, 5, 6, 0, 0]).view(3, 5)
    t = sum(lens)
    x = torch.randn((t, hq + 2 * h, d), generator=g).to(dtype).to(DEV)
    qo, ko = Guarded((t, hq, d), dtype, DEV, seed=6), Guarded((t, h, d), dtype, DEV, seed=7)
    sq.sq_rope_kv_append(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], cache, pages, ints([0, 0, 0]), ints([0, 70, 70, 103]), table=table.t,
                         q_out=qo.t, k_out=ko.t)
    for b in (*codes, *scales, qo, ko):
        b.check("rope_kv_append")
    kr, vr = Guarded((t, h, d), dtype, DEV, seed=8), Guarded((t, h, d), dtype, DEV, seed=9)
    sq.sq_kv_read(cache, pages, ints([0, 0, 0]), ints([0, 70, 70, 103]), t, k_out=kr.t, v_out=vr.t)
    kr.check("kv_read k")
    vr.check("kv_read v")
    q = torch.randn((3, l, hq, d), generator=g).to(dtype).to(DEV)
    out, lse = Guarded((3, l, hq, d), dtype, DEV, seed=10), Guarded((3, l, hq), torch.float32, DEV, seed=11)
    ws = Guarded((sq.sq_kv_attention_workspace_size(cache, 3, l, hq),), torch.uint8, DEV, seed=12)
    sq.sq_kv_attention(q, cache, pages, ints(lens), out=out.t, lse=lse.t, workspace=ws.t)
    for b in (out, lse, ws, *codes, *scales):
        b.check("kv_attention")
    xb = x.bfloat16()
    po, pl = Guarded((t, hq, d), torch.bfloat16, DEV, seed=13), Guarded((t, hq), torch.float32, DEV, seed=14)
    sq.sq_prompt_attention(xb[:, :hq], xb[:, hq:hq + h], xb[:, hq + h:], ints([0, 70, 70, 103]), out=po.t, lse=pl.t)
    po.check("prompt_attention out")
    pl.check("prompt_attention lse")
    assert sq.sq_get_status() == sq.SQ_OK


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, many times."""
    g = torch.Generator().manual_seed(3)
    cache = sq.KvCache.empty(64, 2, 128, page_size=16, scale_block=16)
    x = torch.randn((900, 4, 128), generator=g).bfloat16().to(DEV)
    pages = torch.arange(64, dtype=torch.int32, device=DEV).view(1, 64)
    sq.sq_rope_kv_append(None, x[:, :2], x[:, 2:], cache, pages, ints([0]), ints([0, 900]))
    q = [torch.randn((1, 1, 16, 128), generator=g).bfloat16().to(DEV) for _ in range(2)]
    n = [ints([900]), ints([333])]
    want = [sq.sq_kv_attention(q[i], cache, pages, n[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(sq.sq_kv_attention(q[i], cache, pages, n[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    assert sq.sq_get_status() == sq.SQ_OK


def test_largest_row_counts_and_many_sequences():
    """128 rows of one head, 300 sequences of one or no token."""
    cache = sq.KvCache.empty(300, 1, 64, page_size=16, scale_block=1)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((300, 2, 64), generator=g).to(DEV)
    pages = torch.arange(300, dtype=torch.int32, device=DEV).view(300, 1)
    cu = torch.arange(301, dtype=torch.int32, device=DEV)
    sq.sq_rope_kv_append(None, x[:, :1], x[:, 1:], cache, pages, torch.zeros(300, dtype=torch.int32, device=DEV), cu)
    lens = (torch.arange(300, device=DEV) % 3 > 0).int()
    out, lse = sq.sq_kv_attention(torch.randn((300, 1, 128, 64), generator=g).to(DEV), cache, pages, lens, want_lse=True)
    v, _ = sq.sq_kv_read(cache, pages, ints([0] * 300), cu, 300, dtype=torch.float32), None
    want = torch.where(lens[:, None, None] > 0, v[1], 0.0).expand(300, 128, 64)
    assert (out[:, 0] - want).abs().max() <= 2.0 ** -20 * want.abs().max()
    assert torch.isneginf(lse[lens == 0]).all() and torch.isfinite(lse[lens == 1]).all()
    assert sq.sq_get_status() == sq.SQ_OK


def _soon_overwritten(nbytes):
    """Leave the allocator a block of nbytes that the current stream is still to write."""
    x = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(100_000_000)
    x.fill_(0x7b)


def test_results_for_a_named_stream_are_not_on_the_current_streams_memory():
    """The caller's stream has work before it that writes memory freed since; a call on another stream,
    which does not wait for that work, must not get this memory for its result or workspace."""
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    want = sq.sq_rope_table(4096, 128)
    torch.cuda.synchronize()
    _soon_overwritten(want.numel() * 4)
    for stream in (side, side.cuda_stream):
        got = sq.sq_rope_table(4096, 128, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)

    h, d, n = 8, 128, 2048
    cache = sq.KvCache.empty(n // 64, h, d)
    g = torch.Generator().manual_seed(5)
    x = torch.randn((n, 2 * h, d), generator=g).bfloat16().to(DEV)
    pages, zero, cu, lens = torch.arange(n // 64, dtype=torch.int32, device=DEV).view(1, -1), ints([0]), ints([0, n]), ints([n])
    sq.sq_rope_kv_append(None, x[:, :h], x[:, h:], cache, pages, zero, cu)
    want = sq.sq_kv_read(cache, pages, zero, cu, n)
    torch.cuda.synchronize()
    for _ in range(2):
        _soon_overwritten(n * h * d * 2)
    got = sq.sq_kv_read(cache, pages, zero, cu, n, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sq.sq_get_status() == sq.SQ_OK


def test_a_result_for_a_named_stream_is_kept_while_the_caller_reads_it():
    """Freed by the caller with a read of it still to run on the current stream: its memory is not
    given to the named stream's next result before that."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = sq.sq_rope_table(4096, 128)
    for _ in range(3):
        t = sq.sq_rope_table(4096, 128, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(50_000_000)
        copy = t.clone()
        del t
        other = sq.sq_rope_table(4096, 128, first_pos=77, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del other
    assert sq.sq_get_status() == sq.SQ_OK


@pytest.mark.parametrize("handle", [False, True])
def test_all_calls_on_a_named_stream(handle):
    """The same results as on the current stream, whose memory is about to be overwritten; the
    default stream named while another is the current one."""
    lens, hq, h, d = [70, 33], 6, 2, 64
    t = sum(lens)
    g = torch.Generator().manual_seed(7)
    x = torch.randn((t, hq + 2 * h, d), generator=g).bfloat16().to(DEV)
    pages, zero, cu, n = ints(range(10)).view(2, 5), ints([0, 0]), ints([0, 70, 103]), ints(lens)

    def calls(stream):
        cache = sq.KvCache(*(c.clone() for c in blank))
        torch.cuda.synchronize()
        if stream is not None:
            for size in (96 * 32 * 8, t * hq * d * 2, t * h * d * 2, 4_000_000):
                _soon_overwritten(size)
        table = sq.sq_rope_table(96, d, stream=stream)
        q, k = sq.sq_rope_kv_append(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], cache, pages, zero, cu, table=table, want_k=True, stream=stream)
        kr, vr = sq.sq_kv_read(cache, pages, zero, cu, t, stream=stream)
        a, al = sq.sq_kv_attention(q[[69, 102]].view(2, 1, hq, d) if stream is None else last, cache, pages, n, want_lse=True, stream=stream)
        p, pl = sq.sq_prompt_attention(q, k, x[:, hq + h:], cu, want_lse=True, stream=stream)
        torch.cuda.synchronize()
        return table, q, k, kr, vr, a, al, p, pl, *cache

    side = torch.cuda.Stream()
    blank = sq.KvCache.empty(10, h, d, page_size=16, scale_block=4)
    for c in blank:
        c.zero_()
    want = calls(None)
    last = want[1][[69, 102]].view(2, 1, hq, d)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(calls(side.cuda_stream if handle else side), want))
    assert all(torch.equal(a, b) for a, b in zip(calls(torch.cuda.current_stream()), want))
    with torch.cuda.stream(side):
        got = calls(0 if handle else torch.cuda.default_stream())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sq.sq_get_status() == sq.SQ_OK


def test_a_named_stream_inside_a_capture():
    cache = sq.KvCache(*(c.zero_() for c in sq.KvCache.empty(4, 1, 64, page_size=16, scale_block=16)))
    cache.k_scale.fill_(0.01)
    cache.v.fill_(5)
    cache.v_scale.fill_(0.5)
    pages, n = ints(range(4)).view(1, 4), ints([60])
    q = torch.randn((1, 1, 4, 64), device=DEV)
    sq.sq_kv_attention(q, cache, pages, n)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a = sq.sq_kv_attention(q, cache, pages, n, stream=side)
        b = sq.sq_kv_attention(q, cache, pages, n)
        main.wait_stream(side)
    for _ in range(3):
        a.zero_(), b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and (a - 2.5).abs().max() <= 2.5 * 2.0 ** -20
    assert sq.sq_get_status() == sq.SQ_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_most_sequences(dtype):
    """65,536 sequences, most of them empty: a token here and there, one long one, all calls."""
    n, h, hq, d, ps = 65536, 1, 4, 64, 16
    lens = torch.zeros(n, dtype=torch.int64)
    lens[::1000] = 1
    lens[-1] = 300
    lens[12345] = 77
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    t = int(cu[-1])
    need = (lens + ps - 1) // ps
    pages = torch.full((n, 19), -1, dtype=torch.int32)     # never read where a sequence has no token
    order = torch.randperm(int(need.sum()), generator=torch.Generator().manual_seed(1)).int()
    at = 0
    for b in torch.nonzero(need).flatten().tolist():
        pages[b, :need[b]] = order[at:at + int(need[b])]
        at += int(need[b])
    pages, cu, lens, zero = pages.to(DEV), cu.to(DEV), lens.int().to(DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((t, hq + 2 * h, d), generator=g).to(dtype).to(DEV)
    cache = sq.KvCache.empty(len(order), h, d, page_size=ps, scale_block=1)
    q, k = sq.sq_rope_kv_append(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], cache, pages, zero, cu, want_k=True)
    assert torch.equal(q, x[:, :hq]) and torch.equal(k, x[:, hq:hq + h])
    kr, vr = sq.sq_kv_read(cache, pages, zero, cu, t, dtype=torch.float32)
    step = x[:, hq:].float().abs().amax(-1, keepdim=True) / 127
    assert ((kr - x[:, hq:hq + h].float()).abs() <= 0.5001 * step[:, :h]).all()
    assert ((vr - x[:, hq + h:].float()).abs() <= 0.5001 * step[:, h:]).all()
    last = torch.zeros((n, 1, hq, d), dtype=dtype, device=DEV)
    has = lens > 0
    last[has, 0] = q[(cu[1:][has] - 1).long()]
    out, lse = sq.sq_kv_attention(last, cache, pages, lens, want_lse=True)
    assert not out[~has].any() and torch.isneginf(lse[~has]).all() and torch.isfinite(lse[has]).all()
    xb = x.bfloat16()
    prompt = sq.sq_prompt_attention(xb[:, :hq], xb[:, hq:hq + h], xb[:, hq + h:], cu)
    assert sq.sq_get_status() == sq.SQ_OK
    f32 = dtype == torch.float32
    host = [y.float().cpu().numpy() for y in (q, kr, vr, xb)]
    out, prompt = out.float().cpu().numpy(), prompt.float().cpu().numpy()
    for b in torch.nonzero(has).flatten().tolist():
        a, e = int(cu[b]), int(cu[b + 1])
        seen = np.ones((hq, e - a), bool)
        want, _, bound, _ = ref.attention(host[0][e - 1], host[1][a:e, 0], host[2][a:e, 0], d ** -0.5, seen,
                                          2.0 ** -22 if f32 else 2.0 ** -11, 2.0 ** -24 if f32 else 2.0 ** -8, q_step=2.0 ** -24)
        assert np.all(np.abs(out[b, 0] - want) <= bound)
        want, _, bound, _ = ref.attention(host[3][e - 1, :hq], host[3][a:e, hq], host[3][a:e, hq + h], d ** -0.5, seen, 2.0 ** -8, 2.0 ** -8)
        assert np.all(np.abs(prompt[e - 1] - want) <= bound)
