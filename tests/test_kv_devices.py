"""Which CUDA device the attention over the cache asks for its workspace's size
and runs on, with stand-ins for the tensors and the library; an output without
its input is refused (CPU only)."""
import contextlib
import types

import pytest
import torch


class Standin:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index

    is_cuda = True

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def new_empty(self, shape, dtype):
        return Standin(shape, dtype, self.index)


@pytest.mark.parametrize("current,own", [(0, 0), (0, 1), (1, 0)])
def test_the_workspace_is_sized_on_the_caches_device(monkeypatch, current, own):
    from w8a8_post_quantization_calibrate_b200 import build
    build.build()
    from w8a8_post_quantization_calibrate_b200 import sq
    at = [current]
    sizes = {0: 4096, 1: 8192}
    calls = []

    @contextlib.contextmanager
    def device(index):
        before, at[0] = at[0], index
        yield
        at[0] = before

    def attention(*args):
        calls.append((at[0], args[14]))
        return sq.SQ_OK

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(sq, "_lib", types.SimpleNamespace(
        sq_kv_attention_workspace_size=lambda *args: sizes[at[0]], sq_kv_attention=attention))
    codes, scales = Standin((4, 2, 16, 64), torch.int8, own), Standin((4, 2, 1), torch.float32, own)
    cache = sq.KvCache(codes, codes, scales, scales)
    sq.sq_kv_attention(Standin((3, 1, 8, 64), torch.bfloat16, own), cache, Standin((3, 2), torch.int32, own),
                       Standin((3,), torch.int32, own))
    assert calls == [(own, sizes[own])]
    assert sq.sq_kv_attention_workspace_size(cache, 3, 1, 8) == sizes[own]
    assert at == [current]


def test_a_rotated_q_needs_a_q(monkeypatch):
    from w8a8_post_quantization_calibrate_b200 import build
    build.build()
    from w8a8_post_quantization_calibrate_b200 import sq
    monkeypatch.setattr(sq, "_lib", types.SimpleNamespace())   # nothing to launch
    codes, scales = Standin((4, 2, 16, 64), torch.int8, 0), Standin((4, 2, 1), torch.float32, 0)
    x = Standin((3, 2, 64), torch.bfloat16, 0)
    with pytest.raises(ValueError, match="q_out"):
        sq.sq_rope_kv_append(None, x, x, sq.KvCache(codes, codes, scales, scales), Standin((1, 1), torch.int32, 0),
                             Standin((1,), torch.int32, 0), Standin((2,), torch.int32, 0), q_out=Standin((3, 4, 64), torch.bfloat16, 0))
