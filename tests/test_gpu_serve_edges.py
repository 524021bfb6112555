"""Cache append, paged attention and adapters on the GPU where their numbers
are hard: weak keys beside a strong one, very long rows, infinities, the same
slot twice, and the accuracy that the kernels claim."""
import numpy as np
import pytest
import torch

import serve_ref as ref
from test_gpu_serve import TYPES, Case, _lora_inputs, _num, _tq

pytestmark = pytest.mark.gpu


def _cache(kind, k, v, page=64):
    """One sequence of the rows of k and v ([tokens][kv_heads][d]), in pages in order."""
    shape = (k.shape[0] // page, page) + tuple(k.shape[1:])
    k, v = (x.view(shape).to(TYPES[kind]).cuda() for x in (k, v))
    return _tq().KvCache(k, v, torch.arange(shape[0], dtype=torch.int32, device="cuda").view(1, -1))


def _rows(m, last):
    """Positions and sequences of m rows that see keys 0 .. last of sequence 0."""
    pos = torch.full((m,), last, dtype=torch.int32, device="cuda")
    return pos, torch.zeros_like(pos)


# ---- append --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m", [6, 640])
def test_append_to_the_same_slot(kind, m):
    """Tokens that share a slot: each feature of its key and value is one of theirs, every other slot is as it was, and
    the queries are each token's own."""
    tq = _tq()
    hq, hk, d, page = 6, 3, 64, 16
    cache = _cache(kind, torch.zeros((64, hk, d)), torch.zeros((64, hk, d)), page)
    qkv = torch.from_numpy(np.random.default_rng(m).normal(size=(m, (hq + 2 * hk) * d)).astype(np.float32)).cuda()
    pos, seq = _rows(m, 37)
    pos[0] = 5  # and one that has its own
    q = tq.tq_kv_append(cache, qkv, hq, pos, None, seq=seq)
    x = qkv.view(m, hq + 2 * hk, d)
    assert torch.equal(q, x[:, :hq].to(q.dtype))
    for c, new in ((cache.k, x[:, hq:hq + hk]), (cache.v, x[:, hq + hk:])):
        new = new.to(c.dtype).float()
        c = c.float()
        assert torch.equal(c[0, 5], new[0])
        assert (c[37 // page, 37 % page] == new[1:]).any(dim=0).all()
        c[0, 5] = c[37 // page, 37 % page] = 0.0
        assert c.count_nonzero() == 0


def test_append_e4m3_scales_at_the_ends_of_binary32():
    """Values at and next to every tie between e4m3 values, for scales whose values or reciprocals are subnormal: the
    byte nearest to the exact quotient."""
    tq = _tq()
    scales = np.array([2.0 ** -125 * 1.0613, 2.0 ** -126.5 * 1.077, 2.0 ** -127.5 * 1.07, 2.0 ** -101, 2.0 ** 126.9, 2.0 ** 127.8],
                      dtype=np.float32)
    ties = np.array([(8 + i + 0.5) * 2.0 ** j for i in range(8) for j in range(-12, 6)])
    d, rows = 64, 12
    x = np.zeros((rows, 3, len(scales), d), dtype=np.float32)
    for h, s in enumerate(scales):
        mid = (ties * float(s))[ties * float(s) < 3e38].astype(np.float32)
        near = [mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(np.inf))]
        near = np.resize(np.stack(near + [-near[1]], 1).ravel(), rows * d).reshape(rows, d)
        x[:, 1, h] = x[:, 2, h] = near
    cache = _cache("e4m3", torch.zeros((64, len(scales), d)), torch.zeros((64, len(scales), d)))
    s_d = torch.from_numpy(scales).cuda()
    cache = tq.KvCache(cache.k, cache.v, cache.pages, s_d, s_d)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    tq.tq_kv_append(cache, torch.from_numpy(x.reshape(rows, -1)).cuda(), len(scales), pos, None, seq=torch.zeros_like(pos))
    want = ref.round_e4m3(x[:, 1].astype(np.float64) / scales.astype(np.float64)[:, None])
    for c in (cache.k, cache.v):
        assert np.array_equal(_num(c[0, :rows]), want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("hq,hk,d,rot,inter", [(3, 3, 64, 64, False), (20, 4, 128, 128, True), (8, 1, 256, 64, False)])
def test_append_of_many_tokens(kind, hq, hk, d, rot, inter):
    """A prompt in which blocks take whole tokens, from half as many tokens as there are blocks at once to several per
    block, with padded rows and indices out of range among the others."""
    tq = _tq()
    at_once = torch.cuda.get_device_properties(0).multi_processor_count * (5 if kind == "e4m3" else 7)
    n, page = 4224, 32
    rng = np.random.default_rng(hq)
    table = rng.permutation(n // page).astype(np.int32)
    freq = np.exp(-rng.uniform(0, 14, rot // 2))
    scale = (rng.uniform(0.5, 1.5, hk) / 100).astype(np.float32)
    i = np.arange(rot // 2)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    for m in (at_once // 2 - 1, at_once // 2, at_once // 2 + 1, at_once, at_once + 1, 2 * at_once + 7, 4096):
        pos = rng.permutation(n)[:m].astype(np.int32)
        seq = np.zeros(m, dtype=np.int32)
        bad = rng.permutation(m)[:40]
        pos[bad[:16]] = -1
        seq[bad[16:24]], seq[bad[24:32]], pos[bad[32:]] = -1, 1, n + bad[32:]
        live = np.ones(m, dtype=bool)
        live[bad] = False
        x = rng.normal(size=(m, hq + 2 * hk, d)).astype(np.float32)
        k, v = (torch.zeros((n // page, page, hk, d)).to(TYPES[kind]).cuda() for _ in range(2))
        s_d = torch.from_numpy(scale).cuda() if kind == "e4m3" else None
        cache = tq.KvCache(k, v, torch.from_numpy(table).cuda().view(1, -1), s_d, s_d)
        ws = tq.workspace(tq.tq_kv_append_workspace())
        q = tq.tq_kv_append(cache, torch.from_numpy(x.reshape(m, -1)).cuda(), hq, torch.from_numpy(pos).cuda(),
                            torch.from_numpy(freq).cuda(), inter, torch.from_numpy(seq).cuda(), ws=ws)
        assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
        turned = x.astype(np.float64)
        angle = pos[:, None, None] * freq
        c, s, e = np.cos(angle), np.sin(angle), turned[:, :hq + hk]
        e[..., lo], e[..., hi] = e[..., lo] * c - e[..., hi] * s, e[..., lo] * s + e[..., hi] * c
        size = ref.rotation_size(x[:, :hq + hk].astype(np.float64), rot // 2, inter) * 2.0 ** -21  # as in _check_append
        turned[pos < 0, :hq], size[pos < 0, :hq] = 0.0, 0.0
        half = torch.finfo(q.dtype).eps / 2
        tiny = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
        assert (np.abs(_num(q) - turned[:, :hq]) <= np.abs(turned[:, :hq]) * half + size[:, :hq] * 1.01 + tiny).all(), m
        for got, new, far in ((k, turned[:, hq:hq + hk], size[:, hq:]), (v, turned[:, hq + hk:], 0.0)):
            got = _num(got).reshape(n, hk, d)
            at = table[pos[live] // page] * page + pos[live] % page
            if kind == "e4m3":
                assert np.array_equal(got[at], ref.round_e4m3(new[live] / scale.astype(np.float64)[:, None])), m
            else:
                far = far[live] * 1.01 if isinstance(far, np.ndarray) else far
                assert (np.abs(got[at] - new[live]) <= np.abs(new[live]) * half + far + tiny).all(), m
            rest = np.ones(n, dtype=bool)
            rest[at] = False
            assert (got[rest] == 0).all(), m


# ---- attention -----------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("gap", [16.0, 18.0, 20.0])
def test_attention_many_weak_keys_beside_a_strong_one(kind, gap):
    """16383 equal keys whose scores are `gap` below one key's, in as many items as there are warps, so that one warp
    has all of a row.  The strong key's value is 0: the output is what the weak ones leave of theirs."""
    tq = _tq()
    n, d, hk, m = 16384, 64, 8, 148
    k, v = torch.zeros((n, hk, d)), torch.full((n, hk, d), 32.0)
    k[5], v[5] = gap, 0.0
    cache = _cache(kind, k, v)
    pos, seq = _rows(m, n - 1)
    out = tq.tq_attn(cache, torch.ones((m, hk, d), dtype=cache.q_dtype).cuda(), pos, 1 / d, seq, out_dtype=tq.TQ_F16)
    w = (n - 1) * np.exp(-gap)
    want = 32.0 * w / (1.0 + w)
    # the output's rounding (2^-11 and half of fp16's smallest step); binary32 running sums: 4096 additions of a lane
    # at 2^-24 of the total, and their exponentials
    bound = want * (2.0 ** -11 + 4096 * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -25
    assert float((out.double() - want).abs().max()) <= bound


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d,hq,hk", [(64, 8, 4), (128, 8, 2), (256, 12, 1)])
def test_attention_weights_keep_32_bits(kind, d, hq, hk):
    """Rows of a few keys with fp16 output: nothing but the output's rounding, the scores' binary32 sums and 2^-20 for
    exponentials, weights and sums."""
    tq = _tq()
    c = Case(d, kind, d, hq, hk, 16, [int(x) for x in np.random.default_rng(d).integers(2, 90, 24)])
    q = c.queries(5)
    got = _num(tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d, out_dtype=tq.TQ_F16))
    K, V = c.values()
    qn, grp = _num(q), hq // hk
    for i in range(c.m):
        j = np.arange(int(c.pos[i]) + 1)
        at = c.table[c.seq[i], j // c.page], j % c.page
        for h in range(hk):
            sl = slice(h * grp, (h + 1) * grp)
            want, size, score = ref.attention(qn[i, sl], K[at][:, h], V[at][:, h], d ** -0.5)
            bound = np.abs(want) * 2.0 ** -11 + size * (2 * score * (d / 16 + 8) * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -25
            assert (np.abs(got[i, sl] - want) <= bound).all(), (i, h)


@pytest.mark.parametrize("kind", list(TYPES))
def test_attention_sums_over_a_million_keys(kind):
    """Equal weights over 2^20 keys, in as many items as there are warps: the output is the mean of the values."""
    tq = _tq()
    n, d, hk, m = 1 << 20, 64, 8, 148
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.empty((n // 64, 64, hk, d), dtype=torch.float16, device="cuda").uniform_(0.5, 1.0, generator=g).to(TYPES[kind])
    cache = tq.KvCache(torch.zeros_like(v), v, torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1))
    pos, seq = _rows(m, n - 1)
    out = tq.tq_attn(cache, torch.zeros((m, hk, d), dtype=cache.q_dtype, device="cuda"), pos, 1.0, seq, out_dtype=tq.TQ_F16)
    want = torch.stack([v[:, :, h].double().mean((0, 1)) for h in range(hk)])
    # the output's rounding; 2^15 or 2^16 additions of a tile's share, each rounded to nearest by at most 2^-24 with
    # an error of either sign: 2^8 times that, four times over
    assert float(((out.double() - want).abs() / want).max()) <= 2.0 ** -11 + 4 * 2.0 ** 8 * 2.0 ** -24


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("strong", [2.5, 20.0])
def test_attention_infinite_values(kind, strong):
    """An infinity among the visible values is the output's infinity, down to weights of e^-40 of the largest, and stays
    in its feature and in the rows that see it.  A weight that underflows binary32 (below e^-87) makes it NaN, as 0
    times infinity is."""
    tq = _tq()
    n, d, hk, hq, scale = 4096, 64, 2, 4, 0.125
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((n, hk, d), generator=g), torch.randn((n, hk, d), generator=g)
    v[3, :, 7], v[100, :, 9], v[2000, 1, 11] = float("inf"), -float("inf"), float("inf")
    q = torch.randn((8, hq, d), generator=g)
    k[4], q[:, 1] = strong, 2.0  # query head 1: key 4 is 16 strong (40 or 320) above the rest's middle
    cache = _cache(kind, k, v)
    q = q.to(cache.q_dtype).cuda()
    last = [3, 50, 200, 4095, 2, 99, 100, 2100]
    pos = torch.tensor(last, dtype=torch.int32).cuda()
    got = _num(tq.tq_attn(cache, q, pos, scale, torch.zeros_like(pos), out_dtype=tq.TQ_F16))
    K, V, qn = _num(cache.k).reshape(n, hk, d), _num(cache.v).reshape(n, hk, d), _num(q)
    for i, p in enumerate(last):
        for h in range(hk):
            sl = slice(2 * h, 2 * h + 2)
            want, size, score = ref.attention(qn[i, sl], K[:p + 1, h], V[:p + 1, h], scale)
            s = scale * (qn[i, sl] @ K[:p + 1, h].T)
            gone = s - s.max(axis=1, keepdims=True) < -87.0
            nan = (gone[:, :, None] & np.isinf(V[:p + 1, h])).any(axis=1)
            inf = np.isinf(want) & ~nan
            assert (np.isinf(got[i, sl]) | np.isnan(got[i, sl]))[nan].all(), (i, h)
            assert np.array_equal(got[i, sl][inf], want[inf]), (i, h)
            bound = ref.attention_bound(want, size, score, p + 1, 6.0, torch.float16, cache.k.dtype)
            ok = ~np.isinf(want)
            assert (np.abs(got[i, sl][ok] - want[ok]) <= bound[ok]).all(), (i, h)


def test_attention_of_too_many_tiles():
    """4096 rows of 2^20 keys on 32 key heads (a table that names one page again and again): zeros and the status."""
    tq = _tq()
    m, hk, n = 4096, 32, 1 << 20
    k = torch.zeros((1, 64, hk, 64), dtype=torch.float16, device="cuda")
    cache = tq.KvCache(k, torch.ones_like(k), torch.zeros((1, n // 64), dtype=torch.int32, device="cuda"))
    pos, seq = _rows(m, n - 1)
    q = torch.zeros((m, hk, 64), dtype=torch.float16, device="cuda")
    out = torch.full((m, hk, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = tq.workspace(tq.tq_attn_workspace(cache, m, hk))
    tq.tq_attn(cache, q, pos, 1.0, seq, out=out, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
    assert out.count_nonzero() == 0 and (ws[:65532] == 0).all()
    # with a window they are few: as ever
    ws = tq.workspace(tq.tq_attn_workspace(cache, m, hk))
    tq.tq_attn(cache, q, pos, 1.0, seq, 100, out=out, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_OK and (out == 1).all()


# ---- adapters ------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [20, 300])
def test_lora_infinite_b(kind, m):
    """An infinity in B gives the infinity of its product with A x, also where A x is 2^-41 of the token's largest, and
    stays in its output feature; times an A x of 0 it is NaN."""
    tq = _tq()
    x, a, b, s, ids, y = _lora_inputs(kind, m, 200, 512, 16, 2)
    ids[:] = 1
    a = (a.float() * 64).to(a.dtype)
    x[:, 0], a[1, :, 0], a[1, 5], a[1, 6] = 2.0 ** -10, 0.0, 0.0, 0.0
    a[1, 5, 0] = 2.0 ** -24
    clean = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
    b = b.clone()
    for n, r, v in ((7, 3, float("inf")), (9, 0, -float("inf")), (11, 5, float("inf")), (13, 6, float("inf"))):
        b[1, n, r] = v
    out = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
    h = _num(x) @ _num(a)[1].T
    got = _num(out)
    assert np.array_equal(got[:, 7], np.copysign(np.inf, h[:, 3])) and np.array_equal(got[:, 9], np.copysign(np.inf, -h[:, 0]))
    assert (got[:, 11] == np.inf).all() and np.isnan(got[:, 13]).all()
    keep = [n for n in range(200) if n not in (7, 9, 11, 13)]
    assert torch.equal(out[:, keep], clean[:, keep])


@pytest.mark.parametrize("kind,m,n,k,rank", [
    ("f16", 8, 512, 17408, 128), ("bf16", 8, 512, 17408, 128), ("f16", 300, 512, 17408, 128), ("bf16", 300, 300, 14336, 72),
    ("f16", 1, 1024, 2560, 16), ("bf16", 64, 700, 2560, 64), ("bf16", 1000, 256, 1024, 64), ("f16", 1000, 256, 1024, 24),
])
def test_lora_keeps_32_bits(kind, m, n, k, rank):
    """The adapters' part alone (y = 0), by norms: 1.2e-6.  A tensor core's sum loses up to 2^-23 of itself per MMA, half
    of that on average and two thirds of its final size over a chain, so a chain of 24 loses 24 x 2^-23 / 3 = 9.5e-7 of
    it; the chains of A x have either sign and add up like their parts do.  Both products together: less than sqrt(2)
    times that, and chains of 16 in one of the two in most cases.  (An A x of 16 bits would leave 7.6e-6, and chains of
    136 MMAs over 17408 features gave 2.5e-6.)"""
    tq = _tq()
    x, a, b, s, ids, y = _lora_inputs(kind, m, n, k, rank, 3)
    y.zero_()
    out = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
    want = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for ad in range(3):
        t = (ids == ad).nonzero()[:, 0].cuda()
        want[t] = s[ad].double() * ((x[t].double() @ a[ad].double().T) @ b[ad].double().T)
    assert float((out.double() - want).norm() / want.norm().clamp(min=1e-30)) <= 1.2e-6


def test_lora_prompts_add_small_terms_first():
    """128 ranks of bf16 adapters over 512 features, by norms: 5.5e-7.  By the rule above the products of A x (4 MMAs to
    a sum) lose 1.6e-7 and the 8 MMAs of the largest terms 3.2e-7; all 24 MMAs on the full sum would lose 9.5e-7."""
    tq = _tq()
    for m in (300, 1000):
        x, a, b, s, ids, y = _lora_inputs("bf16", m, 1024, 512, 128, 1)
        ids[:] = 0
        y.zero_()
        out = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
        want = s[0].double() * ((x.double() @ a[0].double().T) @ b[0].double().T)
        assert float((out.double() - want).norm() / want.norm()) <= 5.5e-7


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 20, 300])
def test_lora_terms_of_one_element(kind, m):
    """A x made of two or three products whose bits do not overlap, and B the identity: the output is A x, to 2^-19
    (2^-22 for two fp16 terms, and four sums that lose 2^-22).  A term less leaves 2^-18 (bf16) or 2^-12 (fp16)."""
    tq = _tq()
    rank, k, g = 128, 1024, torch.Generator().manual_seed(m)
    t = TYPES[kind]
    parts, bits = (3, 8) if kind == "bf16" else (2, 11)
    a = torch.zeros((1, rank, k))
    for i in range(parts):
        a[0, :, 37 * i + 5] = (torch.rand(rank, generator=g) + 1) * 2.0 ** (-bits * i)
    x = torch.zeros((m, k))
    x[:, [37 * i + 5 for i in range(parts)]] = 1.0
    a, x, b = a.to(t).cuda(), x.to(t).cuda(), torch.eye(rank).to(t).cuda()[None].contiguous()
    y = torch.zeros((m, rank), device="cuda")
    out = tq.tq_lora(tq.Lora(a, b), x, torch.zeros(m, dtype=torch.int32, device="cuda"), y)
    want = x.double() @ a[0].double().T
    assert float(((out.double() - want).abs() / want).max()) <= 2.0 ** -19


def test_lora_tokens_by_themselves():
    """A token's output has the same bits wherever it stands among tokens of its adapter that fill the same tiles."""
    tq = _tq()
    for m in (24, 320):
        x, a, b, s, ids, y = _lora_inputs("bf16", m, 200, 1024, 16, 2)
        ids[:] = 1
        lora = tq.Lora(a, b, s)
        out = tq.tq_lora(lora, x, ids.cuda(), y, out=torch.empty_like(y))
        order = torch.randperm(m, generator=torch.Generator().manual_seed(m))
        back = tq.tq_lora(lora, x[order].contiguous(), ids.cuda(), y[order].contiguous())
        assert torch.equal(back, out[order])


# ---- the stack -----------------------------------------------------------------------

def test_stack_steps_of_different_sizes_share_buffers():
    """Steps of 5 and 3 tokens, eager and replayed from a graph, in turn on one set of buffers, give the bits that
    stacks of their own give."""
    import tqsynth
    from decode_matmul_b200.attention import AttentionStack
    tq = _tq()
    shape = tqsynth.StackShape("share-test", 1, 512, 1024, 256, 1536)
    cb = tqsynth.codebook(3)
    cbd = torch.from_numpy(cb.view(np.int16)).cuda()
    host = {op: tqsynth.Weight(3, 0, i, n, k, cb) for i, (op, n, k) in enumerate(shape.ops())}
    layers = [{op: tq.DeviceWeight.from_host(w.codes, w.scales, cbd, w.n, w.k) for op, w in host.items()}]
    cases = [Case(9, "bf16", 128, 8, 2, 16, [40, 3, 17, 30, 9], shuffle_seq=False) for _ in range(3)]
    h = torch.from_numpy(tqsynth.activations(1, 5, 512).view(np.int16)).cuda()
    pos = cases[0].pos_d
    alone = [AttentionStack(layers, [c.cache]).forward(h[:m], pos[:m], 5) for c, m in zip(cases, (5, 3))]
    stack = AttentionStack(layers, [cases[2].cache])
    out5, out3 = torch.empty_like(h), torch.empty_like(h[:3])
    stack.forward(h, pos, 5, out=out5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stack.forward(h[:3], pos[:3], 5, out=out3)
    for _ in range(2):
        out5.zero_()
        out3.zero_()
        g.replay()
        stack.forward(h, pos, 5, out=out5)
        assert torch.equal(out5, alone[0]) and torch.equal(out3, alone[1])
    assert tq.tq_workspace_status(stack.buffers(3)["ws"]) == tq.TQ_OK
