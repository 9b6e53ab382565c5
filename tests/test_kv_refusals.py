"""The cache and attention calls reject bad arguments on the host before any
CUDA call (CPU only)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def sq():
    from w8a8_post_quantization_calibrate_b200 import build
    build.build()
    from w8a8_post_quantization_calibrate_b200 import sq as binding
    return binding


P = ctypes.c_void_p(0x1000)      # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1008)
ST = ctypes.c_void_p(0)


def cache(sq, **over):
    f = dict(k=0x1000, v=0x1000, k_scale=0x1000, v_scale=0x1000, n_pages=10, n_heads=4, head_dim=128, page_size=64, scale_block=16)
    f.update(over)
    return sq._KV_CACHE.pack(*f.values())


BAD_CACHES = [
    (dict(head_dim=96), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"), (dict(page_size=256), "UNSUPPORTED"),
    (dict(scale_block=0), "UNSUPPORTED"), (dict(scale_block=12), "UNSUPPORTED"), (dict(scale_block=128), "UNSUPPORTED"),
    (dict(n_heads=0), "UNSUPPORTED"), (dict(n_heads=2000), "UNSUPPORTED"), (dict(n_pages=-1), "INVALID_ARG"),
    (dict(k=0), "INVALID_ARG"), (dict(v_scale=0), "INVALID_ARG"), (dict(v=0x1008), "UNSUPPORTED"),
]


def append(sq, c=None, table=P, max_pages=8, ctx=P, cu=P, n=2, T=4, q=P, qs=8 * 128, hq=8, k=P, ks=512, v=P, vs=512, dt=None,
           cos=P, n_pos=100, rot=128, qo=P, ko=P):
    return sq.raw_status("sq_rope_kv_append", cache(sq) if c is None else c, table, max_pages, ctx, cu, n, T, q, qs, hq, k, ks,
                         v, vs, sq.SQ_BF16 if dt is None else dt, cos, n_pos, rot, 0, qo, ko, ST)


def read(sq, c=None, table=P, max_pages=8, first=P, cu=P, n=2, T=4, k=P, v=P, dt=1):
    return sq.raw_status("sq_kv_read", cache(sq) if c is None else c, table, max_pages, first, cu, n, T, k, v, dt, ST)


def attend(sq, c=None, table=P, max_pages=8, q=P, qs=8 * 128, dt=1, lens=P, n=2, l=1, hq=8, scale=0.1, out=P, ws=P, wsb=1 << 40):
    return sq.raw_status("sq_kv_attention", q, qs, dt, cache(sq) if c is None else c, table, max_pages, lens, n, l, hq,
                         ctypes.c_float(scale), out, None, ws, wsb, ST)


def prompt(sq, q=P, qs=1024, k=P, ks=512, v=P, vs=512, cu=P, n=2, T=10, hq=8, h=4, d=128, scale=0.1, out=P):
    return sq.raw_status("sq_prompt_attention", q, qs, k, ks, v, vs, cu, n, T, hq, h, d, ctypes.c_float(scale), 1, out, None, ST)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches(sq, over, status):
    want = getattr(sq, "SQ_ERR_" + status)
    assert append(sq, c=cache(sq, **over)) == want
    assert read(sq, c=cache(sq, **over)) == want
    assert attend(sq, c=cache(sq, **over)) == want


def test_bad_append(sq):
    inv, uns = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
    assert sq.raw_status("sq_rope_kv_append", None, P, 1, P, P, 1, 1, P, 512, 4, P, 512, P, 512, 1, P, 1, 128, 0, P, P, ST) == inv
    for kw, want in [(dict(dt=2), uns), (dict(dt=9), uns), (dict(n=-1), inv), (dict(T=-1), inv), (dict(hq=-1), inv),
                     (dict(max_pages=-1), inv), (dict(n=70000), uns), (dict(T=1 << 31), uns), (dict(max_pages=1 << 30), uns),
                     (dict(rot=24), uns), (dict(rot=144), uns), (dict(rot=-16), inv), (dict(cos=None), inv), (dict(ctx=None), inv),
                     (dict(cu=None), inv), (dict(table=None), inv), (dict(k=None), inv), (dict(v=None), inv), (dict(q=None), inv),
                     (dict(qo=None), inv), (dict(k=ODD), uns), (dict(qo=ODD), uns), (dict(cos=ODD), uns), (dict(ks=516), uns),
                     (dict(ks=256), inv), (dict(qs=512), inv), (dict(hq=2000), uns)]:
        assert append(sq, **kw) == want, kw
    assert append(sq, T=0) == sq.SQ_OK and append(sq, n=0) == sq.SQ_OK


def test_bad_read(sq):
    inv, uns = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
    for kw, want in [(dict(dt=2), uns), (dict(T=-1), inv), (dict(n=-1), inv), (dict(first=None), inv), (dict(cu=None), inv),
                     (dict(k=None), inv), (dict(v=ODD), uns), (dict(T=1 << 31), uns), (dict(table=None), inv)]:
        assert read(sq, **kw) == want, kw
    assert read(sq, T=0) == sq.SQ_OK and read(sq, n=0) == sq.SQ_OK


def test_bad_attention(sq):
    inv, uns = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
    for kw, want in [(dict(dt=2), uns), (dict(hq=6), uns), (dict(l=65), uns), (dict(l=-1), inv), (dict(hq=-4), inv),
                     (dict(scale=float("nan")), inv), (dict(scale=float("inf")), inv), (dict(q=None), inv), (dict(q=ODD), uns),
                     (dict(qs=1020), uns), (dict(qs=512), inv), (dict(lens=None), inv), (dict(out=None), inv),
                     (dict(out=ODD), uns), (dict(table=None), inv)]:
        assert attend(sq, **kw) == want, kw
    assert attend(sq, n=0) == sq.SQ_OK and attend(sq, l=0) == sq.SQ_OK and attend(sq, hq=0) == sq.SQ_OK


def test_bad_prompt(sq):
    inv, uns = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
    for kw, want in [(dict(d=96), uns), (dict(h=3), uns), (dict(h=0), uns), (dict(T=-1), inv), (dict(n=-1), inv),
                     (dict(scale=float("nan")), inv), (dict(q=None), inv), (dict(k=ODD), uns), (dict(vs=516), uns), (dict(ks=256), inv),
                     (dict(cu=None), inv), (dict(out=None), inv), (dict(out=ODD), uns), (dict(T=1 << 30), uns), (dict(n=70000), uns)]:
        assert prompt(sq, **kw) == want, kw
    assert prompt(sq, T=0) == sq.SQ_OK and prompt(sq, n=0) == sq.SQ_OK and prompt(sq, hq=0) == sq.SQ_OK


def test_bad_table(sq):
    inv, uns = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED

    def table(out=P, first=0, n=4, rot=128, theta=1e4, sc=None):
        s = None if sc is None else sq._ROPE_SCALING.pack(*sc)
        return sq.raw_status("sq_rope_table", out, first, n, rot, ctypes.c_double(theta), s, ST)

    for kw, want in [(dict(first=-1), inv), (dict(n=-1), inv), (dict(rot=24), uns), (dict(rot=0), uns), (dict(rot=272), uns),
                     (dict(theta=0.0), inv), (dict(theta=float("inf")), inv), (dict(out=None), inv), (dict(out=ODD), uns),
                     (dict(first=2 ** 31), uns), (dict(sc=(0.0, 0, 0, 0, 1.0)), inv), (dict(sc=(2.0, 4.0, 1.0, 100, 1.0)), inv),
                     (dict(sc=(2.0, 1.0, 4.0, 0, 1.0)), inv), (dict(sc=(2.0, 0, 0, 0, float("nan"))), inv)]:
        assert table(**kw) == want, kw
    assert table(n=0) == sq.SQ_OK


def test_the_binding_checks_shapes_before_the_call(sq):
    torch = sq.torch
    with pytest.raises(ValueError, match="CUDA"):
        sq.sq_prompt_attention(*[torch.zeros((4, 2, 64), dtype=torch.bfloat16)] * 3, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="bfloat16"):
        sq.sq_prompt_attention(*[torch.zeros((4, 2, 64))] * 3, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        c = sq.KvCache.empty(2, 1, 64, 16, 16, device="cpu")
        sq.sq_kv_attention(torch.zeros((1, 1, 1, 64)), c, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        sq.sq_rope_table(4, 16, table=torch.zeros((4, 8, 2)))
    with pytest.raises(ValueError, match="CUDA"):
        sq.sq_rope_table(4, 16, device="cpu")
    c = sq.KvCache.empty(2, 1, 64, 16, 16, device="cpu")
    with pytest.raises(ValueError, match="same shapes"):
        sq._cache_bytes(sq.KvCache(c.k, c.v[:1], c.k_scale, c.v_scale))
