"""Argument checks of the cache, attention and adapter calls (no GPU): every
refusal comes before any device call, through the C ABI with fake aligned
addresses that nothing dereferences and through the Python binding with CPU
tensors."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import decode_matmul_b200 as tq
import serve_ref

WS = 1 << 40  # a claimed workspace size that covers any query


def _cache(**kw):
    c = dict(k_d=16, v_d=16, pages_d=16, k_scale_d=None, v_scale_d=None, page_stride=16 * 8 * 128, token_stride=8 * 128,
             head_stride=128, dtype=tq.TQ_BF16, n_pages=10, page_size=16, kv_heads=8, head_dim=128, n_seqs=4, max_pages=5)
    c.update(kw)
    return tq.tq_kv_cache_t(*[c[f] for f, _ in tq.tq_kv_cache_t._fields_])


def _append(cache, **kw):
    a = dict(qkv=16, stride=48 * 128, m=3, heads=32, seq=16, pos=16, freq=16, rot=128, inter=0, out=16, ws=16, n=WS)
    a.update(kw)
    return tq.lib().tq_kv_append(ctypes.byref(cache) if cache is not None else None, a["qkv"], a["stride"], a["m"],
                                 a["heads"], a["seq"], a["pos"], a["freq"], a["rot"], a["inter"], a["out"], a["ws"],
                                 a["n"], None)


def _attn(cache, **kw):
    a = dict(q=16, m=3, heads=32, seq=16, pos=16, scale=0.1, window=0, out=16, t=tq.TQ_BF16, ws=16, n=WS)
    a.update(kw)
    return tq.lib().tq_attn(ctypes.byref(cache) if cache is not None else None, a["q"], a["m"], a["heads"], a["seq"],
                            a["pos"], a["scale"], a["window"], a["out"], a["t"], a["ws"], a["n"], None)


@pytest.mark.parametrize("call", [_append, _attn])
def test_cache_checks(call):
    bad = [(dict(dtype=tq.TQ_F32), tq.TQ_ERR_VALUE), (dict(dtype=9), tq.TQ_ERR_VALUE), (dict(head_dim=80), tq.TQ_ERR_SHAPE),
           (dict(head_dim=0), tq.TQ_ERR_SHAPE), (dict(n_pages=0), tq.TQ_ERR_SHAPE), (dict(page_size=0), tq.TQ_ERR_SHAPE),
           (dict(kv_heads=0), tq.TQ_ERR_SHAPE), (dict(n_seqs=0), tq.TQ_ERR_SHAPE), (dict(max_pages=0), tq.TQ_ERR_SHAPE),
           (dict(page_size=65536, max_pages=32768), tq.TQ_ERR_SHAPE), (dict(k_d=None), tq.TQ_ERR_NULL),
           (dict(v_d=None), tq.TQ_ERR_NULL), (dict(pages_d=None), tq.TQ_ERR_NULL), (dict(k_d=24), tq.TQ_ERR_ALIGN),
           (dict(v_d=18), tq.TQ_ERR_ALIGN), (dict(pages_d=18), tq.TQ_ERR_ALIGN), (dict(page_stride=-8), tq.TQ_ERR_VALUE),
           (dict(token_stride=1028), tq.TQ_ERR_ALIGN), (dict(head_stride=132), tq.TQ_ERR_ALIGN),
           (dict(dtype=tq.TQ_E4M3, head_stride=136), tq.TQ_ERR_ALIGN), (dict(k_scale_d=16), tq.TQ_ERR_VALUE),
           (dict(v_scale_d=16), tq.TQ_ERR_VALUE), (dict(dtype=tq.TQ_E4M3, k_scale_d=18), tq.TQ_ERR_ALIGN)]
    for kw, want in bad:
        assert call(_cache(**kw)) == want, kw
    assert call(None) == tq.TQ_ERR_NULL
    c = _cache()
    for kw, want in [(dict(m=-1), tq.TQ_ERR_SHAPE), (dict(m=4097), tq.TQ_ERR_SHAPE), (dict(heads=0), tq.TQ_ERR_SHAPE),
                     (dict(heads=12), tq.TQ_ERR_SHAPE), (dict(pos=None), tq.TQ_ERR_NULL), (dict(out=None), tq.TQ_ERR_NULL),
                     (dict(pos=18), tq.TQ_ERR_ALIGN), (dict(seq=18), tq.TQ_ERR_ALIGN), (dict(out=24), tq.TQ_ERR_ALIGN),
                     (dict(ws=None), tq.TQ_ERR_WORKSPACE), (dict(n=65535), tq.TQ_ERR_WORKSPACE),
                     (dict(ws=24), tq.TQ_ERR_ALIGN)]:
        assert call(c, **kw) == want, kw
    assert call(c, m=0, pos=None, out=None, ws=None, n=0) == tq.TQ_OK


def test_append_checks():
    c = _cache()
    for kw, want in [(dict(rot=8), tq.TQ_ERR_SHAPE), (dict(rot=144), tq.TQ_ERR_SHAPE), (dict(rot=-16), tq.TQ_ERR_SHAPE),
                     (dict(inter=2), tq.TQ_ERR_VALUE), (dict(stride=48 * 128 - 4), tq.TQ_ERR_SHAPE),
                     (dict(stride=48 * 128 + 2), tq.TQ_ERR_ALIGN), (dict(qkv=None), tq.TQ_ERR_NULL),
                     (dict(qkv=24), tq.TQ_ERR_ALIGN), (dict(freq=None), tq.TQ_ERR_NULL), (dict(freq=20), tq.TQ_ERR_ALIGN)]:
        assert _append(c, **kw) == want, kw


def test_attn_checks():
    c = _cache()
    for kw, want in [(dict(scale=float("nan")), tq.TQ_ERR_VALUE), (dict(scale=float("inf")), tq.TQ_ERR_VALUE),
                     (dict(window=-1), tq.TQ_ERR_VALUE), (dict(t=tq.TQ_F32), tq.TQ_ERR_VALUE),
                     (dict(t=tq.TQ_E4M3), tq.TQ_ERR_VALUE), (dict(q=None), tq.TQ_ERR_NULL), (dict(q=24), tq.TQ_ERR_ALIGN)]:
        assert _attn(c, **kw) == want, kw
    n = ctypes.c_size_t()
    assert tq.lib().tq_attn_workspace(ctypes.byref(c), 3, 32, None) == tq.TQ_ERR_NULL
    assert tq.lib().tq_attn_workspace(ctypes.byref(c), 5000, 32, ctypes.byref(n)) == tq.TQ_ERR_SHAPE
    assert tq.lib().tq_attn_workspace(ctypes.byref(c), 3, 32, ctypes.byref(n)) == tq.TQ_OK and n.value >= 65536
    assert _attn(c, n=n.value - 1) == tq.TQ_ERR_WORKSPACE


def test_lora_checks():
    def call(l=None, **kw):
        f = dict(a_d=16, b_d=16, scale_d=None, dtype=tq.TQ_BF16, n_adapters=4, rank=16, n=1000, k=1024)
        f.update(l or {})
        s = tq.tq_lora_t(*[f[x] for x, _ in tq.tq_lora_t._fields_])
        a = dict(x=16, m=3, ad=16, y=16, ys=1000, out=16, os=1000, ws=16, n=WS)
        a.update(kw)
        return tq.lib().tq_lora(ctypes.byref(s), a["x"], a["m"], a["ad"], a["y"], a["ys"], a["out"], a["os"], a["ws"],
                                a["n"], None)

    for l, want in [(dict(dtype=tq.TQ_F32), tq.TQ_ERR_VALUE), (dict(dtype=tq.TQ_E4M3), tq.TQ_ERR_VALUE),
                    (dict(n_adapters=0), tq.TQ_ERR_SHAPE), (dict(rank=0), tq.TQ_ERR_SHAPE), (dict(rank=12), tq.TQ_ERR_SHAPE),
                    (dict(rank=136), tq.TQ_ERR_SHAPE), (dict(n=0), tq.TQ_ERR_SHAPE), (dict(k=256), tq.TQ_ERR_SHAPE),
                    (dict(k=1000), tq.TQ_ERR_SHAPE), (dict(a_d=None), tq.TQ_ERR_NULL), (dict(b_d=None), tq.TQ_ERR_NULL),
                    (dict(a_d=24), tq.TQ_ERR_ALIGN), (dict(b_d=24), tq.TQ_ERR_ALIGN), (dict(scale_d=18), tq.TQ_ERR_ALIGN)]:
        assert call(l) == want, l
    for kw, want in [(dict(m=-1), tq.TQ_ERR_SHAPE), (dict(m=4097), tq.TQ_ERR_SHAPE), (dict(ys=999), tq.TQ_ERR_SHAPE),
                     (dict(os=999), tq.TQ_ERR_SHAPE), (dict(x=None), tq.TQ_ERR_NULL), (dict(ad=None), tq.TQ_ERR_NULL),
                     (dict(y=None), tq.TQ_ERR_NULL), (dict(out=None), tq.TQ_ERR_NULL), (dict(x=24), tq.TQ_ERR_ALIGN),
                     (dict(y=18), tq.TQ_ERR_ALIGN), (dict(ad=18), tq.TQ_ERR_ALIGN), (dict(ws=None), tq.TQ_ERR_WORKSPACE),
                     (dict(n=65535), tq.TQ_ERR_WORKSPACE), (dict(m=0, x=None), tq.TQ_OK)]:
        assert call(None, **kw) == want, kw


def test_binding_refuses_wrong_tensors():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    pages = torch.zeros((2, 3), dtype=torch.int32)
    tq.KvCache(k, k.clone(), pages)
    for bad in (lambda: tq.KvCache(k, k[:3], pages), lambda: tq.KvCache(k.float(), k.float(), pages),
                lambda: tq.KvCache(k, k.half(), pages), lambda: tq.KvCache(k, k, pages.long()),
                lambda: tq.KvCache(k, k, pages[:, ::2]), lambda: tq.KvCache(k, k, pages, torch.ones(3)),
                lambda: tq.KvCache(k.transpose(2, 3), k.transpose(2, 3), pages),
                lambda: tq.KvCache(k, k.transpose(0, 1).contiguous().transpose(0, 1), pages),
                lambda: tq.Lora(torch.zeros(2, 8, 512), torch.zeros(2, 9, 8)),
                lambda: tq.Lora(torch.zeros(2, 8, 512).half(), torch.zeros(2, 9, 16).half()),
                lambda: tq.Lora(torch.zeros(2, 8, 512).half(), torch.zeros(2, 9, 8).half(), torch.ones(3))):
        with pytest.raises(ValueError):
            bad()
    cache = tq.KvCache(k, k.clone(), pages)
    pos = torch.zeros(2, dtype=torch.int32)
    good = torch.zeros((2, (4 + 4) * 64))
    for args in ((good.half(), 4, pos), (good[:, 1:], 4, pos), (good, 4, pos.long()), (good, 4, pos[:1]),
                 (good, 4, pos, torch.ones(16)), (torch.zeros((3, 512)), 4, torch.zeros(3, dtype=torch.int32)),
                 (good, 4, pos)):  # the last one: CPU tensors
        with pytest.raises(ValueError):
            tq.tq_kv_append(cache, *args)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for args in ((q.half(), pos, 1.0), (q[:, :, :32], pos, 1.0), (q, pos[:1], 1.0), (q, pos, 1.0, pos.long()),
                 (q, pos, 1.0)):
        with pytest.raises(ValueError):
            tq.tq_attn(cache, *args)
    lora = tq.Lora(torch.zeros((2, 8, 512), dtype=torch.bfloat16), torch.zeros((2, 9, 8), dtype=torch.bfloat16))
    x, ids, y = torch.zeros((2, 512), dtype=torch.bfloat16), pos, torch.zeros((2, 9))
    for args in ((x.half(), ids, y), (x, ids.long(), y), (x, ids, y[:, :8]), (x, ids, y.double()), (x, ids, y)):
        with pytest.raises(ValueError):
            tq.tq_lora(lora, *args)


def _stack_parts(dtypes=(torch.bfloat16, torch.bfloat16), heads=(2, 2), **sizes):
    """Two layers of weights without bytes (hidden 512, 4 query and 2 key heads of 64, 1024 between) and their caches;
    sizes: what the second layer has instead."""
    shape = dict(q=(256, 512), k=(128, 512), v=(128, 512), o=(512, 256), gate=(1024, 512), up=(1024, 512), down=(512, 1024))
    none = torch.zeros(0)
    layers = [{op: tq.DeviceWeight(none, none, none, *s) for op, s in d.items()} for d in (shape, {**shape, **sizes})]
    caches = [tq.KvCache(torch.zeros((4, 16, n, 64), dtype=t), torch.zeros((4, 16, n, 64), dtype=t),
                         torch.zeros((2, 3), dtype=torch.int32)) for t, n in zip(dtypes, heads)]
    return layers, caches


def test_stack_refusals(monkeypatch):
    """A stack whose layers would not fit its buffers, an output that is not like its input, and a capture before the
    buffers are there."""
    from decode_matmul_b200.attention import AttentionStack
    layers, caches = _stack_parts()
    stack = AttentionStack(layers, caches)
    AttentionStack(*_stack_parts(dtypes=(torch.float16, torch.float8_e4m3fn)))
    for bad in (dict(gate=(2048, 512), up=(2048, 512), down=(512, 2048)), dict(o=(1024, 256)), dict(down=(1024, 1024)),
                dict(q=(512, 512), o=(512, 512)), dict(k=(256, 512), v=(256, 512), heads=(2, 4)),
                dict(dtypes=(torch.float16, torch.bfloat16)), dict(heads=(4, 4)), dict(up=(512, 512))):
        with pytest.raises(ValueError):
            AttentionStack(*_stack_parts(**bad))
    for args in ((layers, caches[:1]), ([], []), (layers, caches, None, False, None, 0, [{}])):
        with pytest.raises(ValueError):
            AttentionStack(*args)
    lora = tq.Lora(torch.zeros((1, 8, 512)).bfloat16(), torch.zeros((1, 128, 8)).bfloat16())
    with pytest.raises(ValueError):
        AttentionStack(layers, caches, adapters=[{"q": lora}, {}])
    h, pos = torch.zeros((2, 512), dtype=torch.int16), torch.zeros(2, dtype=torch.int32)
    for args in ((h.float(), pos), (h[:, :256], pos), (h[0], pos), (h.t().contiguous().t(), pos)):
        with pytest.raises(ValueError):
            stack.forward(*args, 0)
    for out in (h[:1], h.float(), torch.zeros((2, 1024), dtype=torch.int16)[:, :512]):
        with pytest.raises(ValueError):
            stack.forward(h, pos, 0, out=out)
    with pytest.raises(ValueError):  # no adapter indices
        AttentionStack(layers, caches, adapters=[{}, {"k": lora}]).forward(h, pos, 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    with pytest.raises(RuntimeError, match="captured"):
        stack.buffers(2)


def test_plain_forms():
    """The 64-bit forms themselves: e4m3 rounding against torch's cast of every
    fp16 value, the rotation's norm and inverse, attention's limits."""
    x = np.arange(65536, dtype=np.uint16).view(np.float16).astype(np.float64)
    x = x[np.abs(x) <= 448.0]
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(serve_ref.round_e4m3(x), want)
    r = np.random.default_rng(0)
    v, f = r.normal(size=(3, 64)), r.uniform(size=16)
    for inter in (False, True):
        u = serve_ref.rotate(v, 1234.0, f, inter)
        assert np.allclose((u ** 2).sum(1), (v ** 2).sum(1)) and np.array_equal(u[:, 32:], v[:, 32:])
        assert np.allclose(serve_ref.rotate(u, -1234.0, f, inter), v)
    k, vv = r.normal(size=(5, 8)), r.normal(size=(5, 8))
    assert np.allclose(serve_ref.attention(np.zeros((1, 8)), k, vv, 1.0)[0], vv.mean(0))
    assert np.allclose(serve_ref.attention(1e4 * k[2:3], k, vv, 1.0)[0], vv[np.argmax(k @ k[2])])
