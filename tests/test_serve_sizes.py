"""Argument checks and host-side rules of the cache, attention and adapter
calls that need no GPU, where sizes or arguments interact."""
import ctypes

import pytest
import torch

import decode_matmul_b200 as tq


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
