"""Argument checks and host-side rules of the cache, attention and adapter
calls that need no GPU, where sizes or arguments interact."""
import contextlib
import ctypes

import pytest
import torch

import decode_matmul_b200 as tq
from test_serve_args import _stack_parts


def _lora(**kw):
    f = dict(a_d=16, b_d=16, scale_d=None, dtype=tq.TQ_BF16, n_adapters=4, rank=16, n=1000, k=1024)
    f.update(kw)
    return tq.tq_lora_t(*[f[x] for x, _ in tq.tq_lora_t._fields_])


def _lora_workspace(lora, m):
    n = ctypes.c_size_t()
    assert tq.lib().tq_lora_workspace(ctypes.byref(lora), m, ctypes.byref(n)) == tq.TQ_OK
    return n.value


def _call_lora(lora, m, ws_bytes, **kw):
    a = dict(y=16, ys=lora.n, out=16, os=lora.n)
    a.update(kw)
    return tq.lib().tq_lora(ctypes.byref(lora), 16, m, 16, a["y"], a["ys"], a["out"], a["os"], 16, ws_bytes, None)


@pytest.mark.parametrize("rank,k", [(8, 512), (64, 2560), (128, 14336), (24, 1024), (64, 1536)])
def test_lora_workspace_covers_fewer_tokens(rank, k):
    """The query never falls as m grows, and its answer for the most tokens is enough for any number of them."""
    lora = _lora(rank=rank, k=k)
    sizes = [_lora_workspace(lora, m) for m in range(4097)]
    assert sizes == sorted(sizes)
    for m in (1, 256, 257, 1000, 1184, 1185, 2048, 3136, 3137, 4000, 4096):
        # past the workspace check: no device here, or another kind
        assert _call_lora(lora, m, sizes[4096]) in (tq.TQ_ERR_CUDA, tq.TQ_ERR_ARCH) if not torch.cuda.is_available() else True
    assert _call_lora(lora, 3136, 65536) == tq.TQ_ERR_WORKSPACE


def test_lora_in_place_needs_equal_strides():
    """Output rows over other rows of y: refused (one row has no stride)."""
    lora = _lora()
    assert _call_lora(lora, 3, 1 << 40, y=16, out=16, ys=1000, os=1004) == tq.TQ_ERR_SHAPE
    if not torch.cuda.is_available():  # past the checks: no device here, or another kind
        assert _call_lora(lora, 1, 1 << 40, y=16, out=16, ys=1000, os=1004) in (tq.TQ_ERR_CUDA, tq.TQ_ERR_ARCH)
        assert _call_lora(lora, 3, 1 << 40, y=16, out=1 << 30, ys=1000, os=1004) in (tq.TQ_ERR_CUDA, tq.TQ_ERR_ARCH)


def test_attn_refuses_windows_beyond_32_bits():
    """2^32 + 5 would arrive as a window of 5."""
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    cache = tq.KvCache(k, k.clone(), torch.zeros((2, 3), dtype=torch.int32))
    q, pos = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for window in (2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5):
        with pytest.raises(ValueError, match="window"):
            tq.tq_attn(cache, q, pos, 0.1, window=window)


def _adapter(n=128, dtype=torch.bfloat16, device="cpu"):
    return tq.Lora(torch.zeros((1, 8, 512), dtype=dtype, device=device), torch.zeros((1, n, 8), dtype=dtype, device=device))


def test_stack_refuses_what_a_step_could_not_take():
    """Adapters of another type or device, weights on another device, frequencies, windows and scales that the calls of
    a step would refuse: when the stack is made."""
    from decode_matmul_b200.attention import AttentionStack
    layers, caches = _stack_parts()
    AttentionStack(layers, caches, torch.ones(32, dtype=torch.float64), adapters=[{"q": _adapter(256)}, {"v": _adapter()}])
    for lora in (_adapter(dtype=torch.float16), _adapter(device="meta")):
        with pytest.raises(ValueError):
            AttentionStack(layers, caches, adapters=[{}, {"k": lora}])
    far = torch.zeros(0, device="meta")
    for part in ((far, torch.zeros(0), torch.zeros(0)), (torch.zeros(0), far, torch.zeros(0)), (torch.zeros(0), torch.zeros(0), far)):
        other = [layers[0], {**layers[1], "up": tq.DeviceWeight(*part, 1024, 512)}]
        with pytest.raises(ValueError):
            AttentionStack(other, caches)
    for kw in (dict(freq=torch.ones(32)), dict(freq=torch.ones(12, dtype=torch.float64)), dict(freq=torch.ones(40, dtype=torch.float64)),
               dict(freq=torch.ones(8, dtype=torch.float64, device="meta")), dict(window=-1), dict(window=2 ** 31),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            AttentionStack(layers, caches, **kw)


def test_stack_refuses_a_step_before_its_first_launch(monkeypatch):
    """Positions, sequences and adapter indices of the wrong type, size or device, and more tokens than block-table rows
    in any layer: before the buffers are made, so no cache is written."""
    from decode_matmul_b200.attention import AttentionStack
    layers, caches = _stack_parts()
    caches[1] = tq.KvCache(caches[1].k, caches[1].v, torch.zeros((1, 3), dtype=torch.int32))
    stack = AttentionStack(layers, caches, adapters=[{}, {"k": _adapter()}])

    def reached(m):
        raise AssertionError("the step began")

    monkeypatch.setattr(stack, "buffers", reached)
    h, i = torch.zeros((2, 512), dtype=torch.int16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(AssertionError):
        stack.forward(h, i, 0, seq=i, adapter=i)
    for pos, seq, ids in ((i.long(), i, i), (i[:1], i, i), (i, i.long(), i), (i, i[:1], i), (i, i, i.long()), (i, i, i[:1]),
                          (i.to("meta"), i, i), (i, i.to("meta"), i), (i, i, i.to("meta")), (i, None, i)):
        with pytest.raises(ValueError):
            stack.forward(h, pos, 0, seq=seq, adapter=ids)


def test_stack_buffers_stay_bounded(monkeypatch):
    """Every number of tokens in turn holds no more than twice the largest set, each with rows of its own size and a
    workspace that every call of its step takes."""
    from decode_matmul_b200.attention import AttentionStack
    shape = dict(q=(512, 512), k=(128, 512), v=(128, 512), o=(512, 512), gate=(1024, 512), up=(1024, 512), down=(512, 1024))
    some = torch.zeros(16)  # an address: nothing reads it
    layers = [{op: tq.DeviceWeight(some, some, some, *s) for op, s in shape.items()} for _ in range(2)]
    caches = _stack_parts()[1]
    lora = _adapter()
    stack = AttentionStack(layers, caches, adapters=[{"k": lora}, {}])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(tq, "workspace", lambda n, dev: torch.empty(n, dtype=torch.uint8, device=dev))
    held = {}
    for m in [1, 2, 15, 16, 17, 33, 64, 65] + list(range(100, 4097, 111)) + [4096, 3, 2000]:
        b = stack.buffers(m)
        assert stack.buffers(m) is b
        assert b["y"].shape == (m, 768) and b["q"].shape == b["attn"].shape == (m, 8, 64)
        assert [tuple(t.shape) for t in b["hand"]] == [(m, 512), (m, 512), (m, 1024), (m, 512)]
        need = [tq.tq_layer_phase_workspace(s, p, m) for s in stack.structs for p in range(4)]
        need += [tq.tq_attn_workspace(c, m, 8) for c in caches] + [tq.tq_lora_workspace(lora, m), 65536]
        assert b["ws"].numel() >= max(need)
        for t in [b["ws"], b["y"], b["q"], b["attn"]] + b["hand"]:
            assert t.is_contiguous() and t.data_ptr() % 16 == 0
            held[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
    largest = stack.buffers(4096)
    largest = sum(t.untyped_storage().nbytes() for t in [largest["ws"], largest["y"], largest["q"], largest["attn"]] + largest["hand"])
    # the sets of 16, 32, ... 2048 tokens: half, a quarter, ... of the activations; workspaces also hold fixed parts
    fixed = 9 * tq.tq_attn_workspace(caches[0], 1, 8) + 9 * (4 << 20)
    assert sum(held.values()) <= 2 * largest + fixed
    with pytest.raises(tq.TqError):
        stack.buffers(4097)
