"""Where the binding takes memory for a call on an explicit stream: from that stream, kept for the current one."""
import contextlib

import pytest
import torch

CURRENT, SIDE = 11, 22


class OnGpu(torch.Tensor):
    """A host tensor that passes the binding's checks for a CUDA tensor."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.kept_for = stream.cuda_stream


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def abi(monkeypatch):
    from int4_w4a16_group_gb300.build import build
    build()
    from int4_w4a16_group_gb300 import _abi
    now, made = [CURRENT], []

    @contextlib.contextmanager
    def under(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    plain_empty = torch.empty

    def empty(shape, dtype, device):
        t = plain_empty(shape, dtype=dtype).as_subclass(OnGpu)
        t.taken_from, t.kept_for = now[-1], None
        made.append(t)
        return t

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 1 << 10) if name.endswith(("_size", "_create")) else (lambda *a: 0)

    monkeypatch.setattr(_abi, "_lib", Lib())
    monkeypatch.setattr(_abi, "_device", lambda: 0)
    monkeypatch.setattr(_abi, "_raw_stream", lambda device: now[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(now[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    _abi.w4a16_attention_workspace_size.cache_clear()
    yield _abi, made
    _abi.w4a16_attention_workspace_size.cache_clear()


def attention_calls(a):
    i32, i64 = torch.int32, torch.int64
    x, pos, tab = on_gpu(3, 4, 64), on_gpu(3, dtype=i32), on_gpu(9, 32, 2)
    cache = on_gpu(2, 4, 16 * 72, dtype=torch.uint8)
    return {
        "rope_table": (1, lambda s: a.w4a16_rope_table(9, 64, stream=s)),
        "rope": (1, lambda s: a.w4a16_rope(x, pos, tab, stream=s)),
        "kv_read": (2, lambda s: a.w4a16_kv_read(cache, on_gpu(3, dtype=i64), 64, stream=s)),
        "attention": (2, lambda s: a.w4a16_attention(x, cache, on_gpu(1, 2, dtype=i32), on_gpu(1, dtype=i32),
                                                     on_gpu(2, dtype=i32), max_q=3, scale=0.1, stream=s)),
    }


def check_calls(abi, calls):
    a, made = abi
    for name, (count, call) in calls(a).items():
        for stream, source, kept in ((None, CURRENT, None), (FakeStream(CURRENT), CURRENT, None), (CURRENT, CURRENT, None),
                                     (FakeStream(SIDE), SIDE, CURRENT), (SIDE, SIDE, CURRENT), (0, 0, CURRENT)):
            made.clear()
            call(stream)
            assert len(made) == count, name
            for t in made:
                assert t.taken_from == source and t.kept_for == kept, (name, source)


def test_attention_entries(abi):
    check_calls(abi, attention_calls)


def linear_calls(a):
    i32, u = torch.int32, torch.float32
    K, N, T, E = 64, 64, 3, 2
    x, qw, sc = on_gpu(T, K), on_gpu(K // 8, N, dtype=i32), on_gpu(K // 32, N)
    ids, w = on_gpu(T, 2, dtype=i32), on_gpu(T, 2)
    gu, dn = (on_gpu(E, K // 8, N, dtype=i32), on_gpu(E, K // 32, N)), (on_gpu(E, 4, K, dtype=i32), on_gpu(E, 1, K))
    shared = (qw, sc, on_gpu(4, K, dtype=i32), on_gpu(1, K))
    return {
        "quantize": (2, lambda s: a.w4a16_quantize(on_gpu(K, N, dtype=u), stream=s)),
        "dequantize": (1, lambda s: a.w4a16_dequantize(qw, sc, stream=s)),
        "gemm": (1, lambda s: a.w4a16_gemm(x, qw, sc, stream=s)),
        "gemm_swiglu": (1, lambda s: a.w4a16_gemm_swiglu(x, qw, sc, stream=s)),
        "gemm_bf16": (1, lambda s: a.w4a16_gemm_bf16(on_gpu(T, K, dtype=torch.bfloat16), qw, sc, stream=s)),
        "moe_gemm": (2, lambda s: a.w4a16_moe_gemm(x, ids, w, *gu, *dn, stream=s)),
        "moe_block": (2, lambda s: a.w4a16_moe_block(x, ids, w, *gu, *dn, *shared, stream=s)),
        "moe_gemm_noalloc": (1, lambda s: a.w4a16_moe_gemm_noalloc(x, ids, w, *gu, *dn, stream=s)),
        "topk_softmax": (1, lambda s: a.w4a16_topk_softmax(w, stream=s)),
    }


def test_linear_and_moe_entries(abi):
    check_calls(abi, linear_calls)


def test_registry_entries(abi, monkeypatch):
    a, _ = abi
    monkeypatch.setattr(a.Registry, "find", lambda self, name: (64, 64))
    r, x = a.Registry(), on_gpu(3, 64)
    try:
        check_calls(abi, lambda a: {"linear": (1, lambda s: r.linear("w", x, stream=s)),
                                    "linear_swiglu": (1, lambda s: r.linear_swiglu("w", x, stream=s))})
    finally:
        r.close()           # its handle is not the library's
