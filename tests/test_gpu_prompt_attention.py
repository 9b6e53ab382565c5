"""Attention of packed prompts over themselves, against 64 bits
(tests/kv_reference.py)."""
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


def check(q, k, v, lens, out, lse, scale, causal):
    hq, h = q.shape[1], k.shape[1]
    q, k, v = (x.float().cpu().numpy() for x in (q, k, v))
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    at = cu_of(lens)
    for a, b in zip(at, at[1:]):
        n = b - a
        seen = np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)
        for j in range(hq):
            jk = j // (hq // h)
            want, wlse, bound, lbound = ref.attention(q[a:b, j], k[a:b, jk], v[a:b, jk], scale, seen, 2.0 ** -8, 2.0 ** -8)
            err = np.abs(out[a:b, j] - want)
            assert np.all(err <= bound), f"rows {a}..{b} head {j}: {np.max(err / bound)} of the bound at {np.argwhere(err > bound)[:3].tolist()}"
            assert np.all(np.abs(lse[a:b, j] - wlse) <= lbound), np.max(np.abs(lse[a:b, j] - wlse) / lbound)


CASES = [
    # lens, hq, h, d
    ([1], 1, 1, 128), ([1, 1, 1], 2, 1, 64), ([127, 128, 129], 2, 2, 128), ([5, 0, 300, 64, 1], 4, 2, 64),
    ([255, 256, 257, 0], 3, 1, 128), ([700], 8, 1, 128), ([1030], 2, 2, 64), ([33] * 30, 4, 4, 128), ([0, 0, 513], 6, 3, 64),
]


def _qkv(t, hq, h, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((t, hq + 2 * h, d), generator=g)
    x[:, hq:hq + h, :2] *= 3.0
    x = x.bfloat16().to(DEV)
    return x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_prompt_attention(case, causal):
    lens, hq, h, d = CASES[case]
    q, k, v = _qkv(sum(lens), hq, h, d, seed=case)
    out, lse = sq.sq_prompt_attention(q, k, v, ints(cu_of(lens)), causal=causal, want_lse=True)
    assert sq.sq_get_status() == sq.SQ_OK
    check(q, k, v, lens, out, lse, d ** -0.5, causal)
    again = sq.sq_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), ints(cu_of(lens)), causal=causal)
    assert torch.equal(out, again), "strided and contiguous inputs differ"


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_scales(scale):
    """Flat, negative and one-hot scores."""
    q, k, v = _qkv(400, 2, 1, 128, seed=1)
    out, lse = sq.sq_prompt_attention(q, k, v, ints([0, 400]), scale=scale, want_lse=True)
    assert sq.sq_get_status() == sq.SQ_OK
    check(q, k, v, [400], out, lse, scale, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_behind_the_last_sequence(d, causal):
    """A padded batch: NaN and infinities in the rows behind the last sequence
    reach nothing, and their outputs stay as they were."""
    lens = [130, 77]
    t = sum(lens)
    q, k, v = (x.clone() for x in _qkv(t + 90, 2, 1, d, seed=3))
    for i, x in enumerate((q, k, v)):
        x[t:] = float("nan") if i != 1 else float("inf")
    out = torch.full((t + 90, 2, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((t + 90, 2), 3.0, device=DEV)
    sq.sq_prompt_attention(q, k, v, ints(cu_of(lens)), causal=causal, out=out, lse=lse)
    assert sq.sq_get_status() == sq.SQ_OK
    check(q[:t], k[:t], v[:t], lens, out[:t], lse[:t], d ** -0.5, causal)
    assert torch.all(out[t:] == 3.0) and torch.all(lse[t:] == 3.0)


@pytest.mark.parametrize("causal", [True, False])
def test_a_neighbour_with_nan_reaches_nothing(causal):
    lens = [70, 140, 33]
    q, k, v = (x.clone() for x in _qkv(sum(lens), 2, 2, 128, seed=4))
    want = sq.sq_prompt_attention(q, k, v, ints(cu_of(lens)), causal=causal)
    for x in (q, k, v):
        x[70:210] = float("nan")
    got = sq.sq_prompt_attention(q, k, v, ints(cu_of(lens)), causal=causal)
    assert torch.equal(got[:70], want[:70]) and torch.equal(got[210:], want[210:])


def test_offsets_outside_the_rows_are_cut_and_reported():
    q, k, v = _qkv(100, 2, 1, 64, seed=5)
    want = sq.sq_prompt_attention(q, k, v, ints([0, 40, 100]))
    got = sq.sq_prompt_attention(q, k, v, ints([0, 40, 150]))
    assert sq.sq_get_status() == sq.SQ_ERR_BOUNDS and sq.sq_get_status() == sq.SQ_OK
    assert torch.equal(got, want)


def test_captured_and_replayed_with_other_lengths():
    q, k, v = (x.contiguous() for x in _qkv(600, 4, 2, 128, seed=6))
    cu = ints([0, 300, 600])
    out = torch.zeros((600, 4, 128), dtype=torch.bfloat16, device=DEV)
    sq.sq_prompt_attention(q, k, v, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.sq_prompt_attention(q, k, v, cu, out=out)
    for lens in ([0, 300, 600], [0, 1, 600], [0, 599, 599]):
        cu.copy_(ints(lens))
        q.neg_()
        want = sq.sq_prompt_attention(q, k, v, cu)
        g.replay()
        assert torch.equal(out[:lens[-1]], want[:lens[-1]])
    assert sq.sq_get_status() == sq.SQ_OK
