"""Where the binding's calls take a workspace from that they are not given: the pool of the stream
they run on (stand-ins for tensors, streams and the library; nothing is launched)."""
import contextlib

import pytest
import torch

from indexer_selected_sparse_block_gb300 import _binding as B

SIDE = type("Stream", (), dict(device_index=0, cuda_stream=77))()


class Fake:
    """What the calls ask of a contiguous CUDA tensor."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = shape, dtype

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return self.dtype.itemsize

    def stride(self, i=None):
        if i is None:
            return tuple(self.stride(k) for k in range(len(self.shape)))
        n = 1
        for s in self.shape[i % len(self.shape) + 1:]:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000


def i32(*s):
    return Fake(*s, dtype=torch.int32)


def f32(*s):
    return Fake(*s, dtype=torch.float32)


Q, K, KP, O = Fake(4, 16, 576), Fake(2, 99, 1, 576), Fake(198, 1, 576), f32(4, 16, 512)
KEPT = (i32(4), i32(4), i32(4, 8), i32(4), 8, 4)
CALLS = {
    "sfa_topk_blocks_refine": lambda s: B.sfa_topk_blocks_refine(
        f32(4, 64), f32(4, 64), Fake(4, 4, 64), f32(4, 4), i32(4), i32(4), Fake(2, 64, 128), 4, 8, 64, i32(4, 8),
        i32(4), stream=s),
    "sfa_topk_blocks": lambda s: B.sfa_topk_blocks(f32(4, 64), i32(4), 4, 8, 64, i32(4, 8), i32(4), stream=s),
    "sfa_gather_attend": lambda s: B.sfa_gather_attend(Q, K, None, *KEPT, 0.1, O, stream=s),
    "sfa_gather_attend_window": lambda s: B.sfa_gather_attend_window(Q, K, None, *KEPT, 16, 0.1, O, stream=s),
    "sfa_dense_attend": lambda s: B.sfa_dense_attend(Q, K, None, i32(4), i32(4), 99, 0.1, O, stream=s),
    "sfa_gather_attend_paged": lambda s: B.sfa_gather_attend_paged(Q, KP, None, i32(2, 99), *KEPT, 0.1, O, stream=s),
    "sfa_dense_attend_paged": lambda s: B.sfa_dense_attend_paged(Q, KP, None, i32(2, 99), i32(4), i32(4), 99, 0.1, O,
                                                                 stream=s),
    "sfa_chunk_attend_paged": lambda s: B.sfa_chunk_attend_paged(Q, KP, None, i32(2, 7), 16, i32(3), i32(2), 2, 99,
                                                                 0.1, O, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [SIDE, None])
def test_workspace_comes_from_the_calls_stream(monkeypatch, name, stream):
    current, taken, launched = ["main"], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, fn):
            def call(*args):
                if fn == name:
                    launched.append(args)
                    return 0
                return 4096                   # the size queries
            call.__name__ = fn
            return call

    def empty(n, dtype=None, device=None):
        taken.append(current[-1])
        return Fake(n, dtype=torch.uint8)

    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(B, "_chunk_workspace", lambda *a: 4096)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SIDE)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 77, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(Fake, "record_stream", lambda self, s: None, raising=False)
    CALLS[name](stream)
    assert len(launched) == 1
    assert taken == ["main" if stream is None else stream]
