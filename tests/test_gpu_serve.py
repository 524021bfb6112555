"""Cache append, paged attention and adapters on the GPU against the plain
64-bit forms of serve_ref.py, at the sizes, masks and layouts where they can go
wrong; refusals that show in the status word; capture, streams and repeats."""
import numpy as np
import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _tq():
    import decode_matmul_b200 as tq
    return tq


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


def _num(t):
    """float64 numpy values of a tensor of any of the types."""
    return t.float().double().cpu().numpy()


class Case:
    """A cache filled with normal values and the pieces around it."""

    def __init__(self, seed, kind, d, q_heads, kv_heads, page, lens, order="ptd", spare=3, junk=None, shuffle_seq=True):
        tq = _tq()
        self.rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        t = TYPES[kind]
        self.kind, self.d, self.hq, self.hk, self.page = kind, d, q_heads, kv_heads, page
        self.m, self.pos = len(lens), np.array([n - 1 for n in lens], dtype=np.int32)
        need = [max(0, -(-n // page)) for n in lens]
        self.width = max(max(need), 1) + 1
        self.n_pages = sum(need) + spare
        ids = self.rng.permutation(self.n_pages)[:sum(need)]
        self.seq = self.rng.permutation(self.m).astype(np.int32) if shuffle_seq else np.arange(self.m, dtype=np.int32)
        # entries behind the last page are out of range: nothing may look at them
        self.table = np.full((self.m, self.width), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[self.seq[i], :n] = ids[at:at + n]
            at += n

        def make():
            x = torch.randn((self.n_pages, page, kv_heads, d), generator=g)
            if kind == "e4m3":
                x = (x * 60).clamp(-448, 448)
            used = torch.zeros((self.n_pages, page), dtype=torch.bool)
            for i, n in enumerate(lens):
                for j in range(n):
                    used[self.table[self.seq[i], j // page], j % page] = True
            if junk is not None:
                x[~used] = junk
            x = x.to(t).cuda()
            if order == "phtd":  # memory [page][head][token][d]
                x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            elif order == "wide":  # strided: every second token row of a wider allocation
                big = torch.zeros((self.n_pages, page, 2, kv_heads, d), dtype=torch.float16).to(t).cuda()
                big[:, :, 1] = x
                x = big[:, :, 1]
            return x

        self.k, self.v = make(), make()
        self.ks = self.vs = None
        if kind == "e4m3":
            self.ks = torch.rand(kv_heads, generator=g).add_(0.5).div_(60).cuda()
            self.vs = torch.rand(kv_heads, generator=g).add_(0.5).div_(60).cuda()
        self.cache = tq.KvCache(self.k, self.v, torch.from_numpy(self.table).cuda(), self.ks, self.vs)
        self.pos_d, self.seq_d = torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.seq).cuda()

    def values(self):
        """(K, V) float64 [page][token][head][d], scales applied."""
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            x = _num(x)
            out.append(x if s is None else x * _num(s)[:, None])
        return out

    def queries(self, seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randn((self.m, self.hq, self.d), generator=g).to(self.cache.q_dtype).cuda()

    def check_attn(self, q, out, scale, window=0, hidden=()):
        """hidden: pages that the call must leave out."""
        K, V = self.values()
        qn, on = _num(q), _num(out)
        grp = self.hq // self.hk
        worst = 0.0
        for i in range(self.m):
            p = int(self.pos[i])
            j = np.arange(max(0, p + 1 - window) if window else 0, p + 1)
            pages = self.table[self.seq[i], j // self.page]
            keep = ~np.isin(pages, list(hidden))
            pages, j = pages[keep], j[keep] % self.page
            for h in range(self.hk):
                sl = slice(h * grp, (h + 1) * grp)
                kk, vv = K[pages, j, h], V[pages, j, h]
                want, size, score = ref.attention(qn[i, sl], kk, vv, scale)
                bound = ref.attention_bound(want, size, score, len(j), np.abs(vv).max() if len(j) else 0.0, out.dtype,
                                            self.k.dtype)
                err = np.abs(on[i, sl] - want)
                assert np.isfinite(on[i, sl]).all(), (i, h)
                if len(j) == 0:
                    assert (on[i, sl] == 0).all(), (i, h)
                else:
                    assert (err <= bound).all(), (i, h, float((err / bound).max()))
                    worst = max(worst, float((err / bound).max()))
        return worst


# ---- append -----------------------------------------------------------------------

APPEND = [  # kind, d, q heads, kv heads, rot, interleaved, page, tokens, memory order
    ("bf16", 128, 32, 8, 128, False, 16, 1, "ptd"),
    ("f16", 128, 4, 4, 128, True, 7, 9, "phtd"),
    ("e4m3", 128, 12, 2, 64, False, 16, 33, "ptd"),
    ("e4m3", 64, 8, 8, 64, True, 1, 20, "phtd"),
    ("bf16", 64, 5, 1, 16, True, 24, 17, "wide"),
    ("f16", 96, 7, 7, 96, False, 100, 5, "ptd"),
    ("e4m3", 96, 14, 2, 48, True, 5, 31, "wide"),
    ("bf16", 256, 16, 1, 256, False, 3, 40, "ptd"),
    ("f16", 256, 3, 3, 0, False, 16, 6, "ptd"),
    ("e4m3", 256, 6, 2, 256, False, 64, 150, "ptd"),
]


@pytest.mark.parametrize("kind,d,hq,hk,rot,inter,page,m,order", APPEND)
def test_append(kind, d, hq, hk, rot, inter, page, m, order):
    tq = _tq()
    rng = np.random.default_rng(m)
    lens = [int(x) for x in rng.integers(1, 70, m)]
    lens[m // 2] = page  # a page that has just become full
    if m > 4:
        lens[3] = 0  # a padded row
    c = Case(m, kind, d, hq, hk, page, lens, order)
    before = [_bytes(c.k), _bytes(c.v)]
    qkv = torch.from_numpy(rng.normal(size=(m, (hq + 2 * hk) * d)).astype(np.float32)).cuda()
    # frequencies with no pattern, up to the largest that is in use
    freq = torch.from_numpy(np.exp(-rng.uniform(0, 14, rot // 2))).cuda() if rot else None
    q = tq.tq_kv_append(c.cache, qkv, hq, c.pos_d, freq, inter, c.seq_d)
    torch.cuda.synchronize()
    _check_append(c, qkv, q, before, freq, inter)


def _check_append(c, qkv, q, before, freq, inter):
    hq, hk, d = c.hq, c.hk, c.d
    x = _num(qkv).reshape(c.m, hq + 2 * hk, d)
    f = _num_f64(freq)
    half = 0 if freq is None else len(f)
    qn, kn, vn = _num(q), _num(c.k), _num(c.v)
    after = [_bytes(c.k), _bytes(c.v)]
    qt = q.dtype
    written = np.zeros((c.n_pages, c.page), dtype=bool)
    for i in range(c.m):
        p = int(c.pos[i])
        if p < 0:
            assert (qn[i] == 0).all()
            continue
        rx = ref.rotate(x[i], float(p), f, inter) if half else x[i]
        # binary32: the sine, the cosine and the reduced angle (2^-22 together),
        # two products and a sum
        size = ref.rotation_size(x[i], half, inter) * 2.0 ** -21 if half else np.zeros_like(x[i])
        slot = (c.table[c.seq[i], p // c.page], p % c.page)
        written[slot] = True
        tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
        assert (np.abs(qn[i] - rx[:hq]) <= np.abs(rx[:hq]) * torch.finfo(qt).eps / 2 + size[:hq] * 1.01 + tiny[qt]).all()
        if c.kind == "e4m3":  # the byte nearest to the exact value
            assert np.array_equal(kn[slot], ref.round_e4m3(rx[hq:hq + hk] / _num(c.ks)[:, None]))
            assert np.array_equal(vn[slot], ref.round_e4m3(x[i, hq + hk:] / _num(c.vs)[:, None]))
        else:
            t = c.k.dtype
            want = rx[hq:hq + hk]
            assert (np.abs(kn[slot] - want) <= np.abs(want) * torch.finfo(t).eps / 2 + size[hq:hq + hk] * 1.01 + tiny[t]).all()
            assert torch.equal(torch.from_numpy(vn[slot]), torch.from_numpy(x[i, hq + hk:]).float().to(t).double())
    for b, a in zip(before, after):  # every other slot is as it was
        assert torch.equal(b[torch.from_numpy(~written)], a[torch.from_numpy(~written)])


def _num_f64(freq):
    return None if freq is None else freq.cpu().numpy()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_far_positions_and_strided_rows(kind):
    """Positions up to 2^31 - 2, where binary32 angles would be noise; rows of a wider buffer."""
    tq = _tq()
    d, hq, hk, page, m = 64, 4, 2, 1024, 6
    c = Case(5, kind, d, hq, hk, page, [page] * m, shuffle_seq=False)
    far = [2 ** 31 - 2, 1_000_003, 2 ** 24 + 1, 131071, 0, 2 ** 30 + 12345]
    width = 2 ** 21 - 1
    table = torch.full((m, width), -1, dtype=torch.int32)
    for i, p in enumerate(far):
        if p // page < width:
            table[i, p // page] = int(c.table[i, 0])
    far[0] = width * page - 1
    table[0, width - 1] = int(c.table[0, 0])
    cache = tq.KvCache(c.k, c.v, table.cuda(), c.ks, c.vs)
    rng = np.random.default_rng(1)
    wide = torch.from_numpy(rng.normal(size=(m, (hq + 2 * hk) * d + 36)).astype(np.float32)).cuda()
    qkv = wide[:, 4:4 + (hq + 2 * hk) * d]
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    pos = torch.tensor(far, dtype=torch.int32).cuda()
    before = [_bytes(c.k), _bytes(c.v)]
    ws = tq.workspace(tq.tq_kv_append_workspace())
    q = tq.tq_kv_append(cache, qkv, hq, pos, freq.cuda(), ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    # the checker's view: the same pages, reached through a table of one page per row
    c.pos = np.array(far, dtype=np.int64)
    c.table = {(i, p // page): int(c.table[i, 0]) for i, p in enumerate(far)}
    _check_append(c, qkv, q, before, freq, False)


def test_append_beyond_32_bit_offsets():
    """Slots past 2^32 elements, in a cache that interleaves k and v by page."""
    tq = _tq()
    d, hk, hq, page = 128, 8, 8, 64
    per = page * hk * d
    n_pages = (2 ** 32) // (2 * per) + 5
    big = torch.empty((n_pages, 2, page, hk, d), dtype=torch.float16, device="cuda")
    k, v = big[:, 0], big[:, 1]
    last = torch.tensor([[n_pages - 1], [0], [n_pages - 2]], dtype=torch.int32, device="cuda")
    for t in (k, v):
        t[n_pages - 2:] = 0
        t[0] = 0
    cache = tq.KvCache(k, v, last)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((3, (hq + 2 * hk) * d), device="cuda", generator=g)
    pos = torch.tensor([63, 0, 5], dtype=torch.int32, device="cuda")
    tq.tq_kv_append(cache, qkv, hq, pos)
    x = qkv.view(3, 3, hq, d).half()
    for i, (pg, j) in enumerate(((n_pages - 1, 63), (0, 0), (n_pages - 2, 5))):
        assert torch.equal(k[pg, j], x[i, 1]) and torch.equal(v[pg, j], x[i, 2])
        assert k[pg].count_nonzero() <= hk * d and v[pg].count_nonzero() <= hk * d
    out = tq.tq_attn(cache, x[:, 0].contiguous(), torch.tensor([63, 0, 5], dtype=torch.int32, device="cuda"), 0.0,
                     out_dtype=tq.TQ_F16)
    # equal weights: the mean of the visible values, of which only the new one is not zero
    for i, n in enumerate((64, 1, 6)):
        want = x[i, 2].double() / n
        assert ((out[i].double() - want).abs() <= want.abs() * 2.0 ** -10 + 2.0 ** -24).all()


def test_append_bad_indices_store_nothing():
    tq = _tq()
    c = Case(2, "bf16", 64, 4, 2, 8, [5] * 6, shuffle_seq=False)
    table = c.cache.pages.clone()
    table[1, 0], table[2, 0] = c.n_pages, -1
    cache = tq.KvCache(c.k, c.v, table)
    pos = torch.tensor([4, 4, 4, 8 * c.width, 4, 2 ** 31 - 1], dtype=torch.int32).cuda()
    seq = torch.tensor([-1, 1, 2, 3, 6, 5], dtype=torch.int32).cuda()
    qkv = torch.randn((6, 8 * 64)).cuda()
    before = [_bytes(c.k), _bytes(c.v)]
    ws = tq.workspace(tq.tq_kv_append_workspace())
    q = tq.tq_kv_append(cache, qkv, 4, pos, None, seq=seq, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
    assert torch.equal(before[0], _bytes(c.k)) and torch.equal(before[1], _bytes(c.v))
    assert torch.equal(q, qkv.view(6, 8, 64)[:, :4].bfloat16())


def test_append_e4m3_extremes():
    """Saturation, NaN, zeros and exact ties."""
    tq = _tq()
    c = Case(2, "e4m3", 64, 1, 1, 8, [1], shuffle_seq=False)
    one = torch.ones(1).cuda()
    cache = tq.KvCache(c.k, c.v, c.cache.pages, one, one)
    v = torch.zeros(64)
    v[:12] = torch.tensor([1e9, -1e9, float("inf"), -float("inf"), 448.0, 464.0, 480.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0,
                           19.0, -0.0])
    qkv = torch.cat([torch.zeros(64), v, v]).view(1, -1).cuda()
    tq.tq_kv_append(cache, qkv, 1, c.pos_d, None)
    page = int(c.table[0, 0])
    want = [448.0, -448.0, 448.0, -448.0, 448.0, 448.0, 448.0, 0.0, 2.0 ** -8, 16.0, 20.0, 0.0]
    for t in (c.k, c.v):
        assert t[page, 0, 0].float()[:12].tolist() == want
    qkv[0, 64], qkv[0, 128] = float("nan"), float("nan")
    tq.tq_kv_append(cache, qkv, 1, c.pos_d, None)
    assert c.k[page, 0, 0].float()[0].isnan() and c.v[page, 0, 0].float()[0].isnan()


# ---- attention -----------------------------------------------------------------------

ATTN = [  # kind, d, q heads, kv heads, page, lengths, window, memory order, out type
    ("bf16", 128, 32, 8, 16, [777], 0, "ptd", "bf16"),
    ("bf16", 128, 8, 8, 16, [1, 15, 16, 17, 31, 32, 33, 0, 128, 129], 0, "phtd", "bf16"),
    ("f16", 64, 20, 4, 24, [1, 2, 200, 0, 401, 95], 0, "ptd", "f16"),
    ("e4m3", 128, 12, 2, 64, [1, 63, 64, 65, 700, 0, 3], 0, "ptd", "bf16"),
    ("f16", 96, 6, 2, 5, [1, 4, 5, 6, 211, 90], 0, "wide", "bf16"),
    ("e4m3", 96, 9, 3, 1, [1, 2, 150, 0], 0, "phtd", "f16"),
    ("bf16", 256, 8, 1, 16, [300, 1, 17], 0, "ptd", "bf16"),
    ("e4m3", 256, 16, 2, 100, [99, 100, 101, 350], 0, "ptd", "bf16"),
    ("f16", 256, 4, 4, 3, [70, 33], 0, "wide", "f16"),
    ("bf16", 64, 16, 1, 16, [500, 20, 1], 0, "ptd", "f16"),
    ("f16", 128, 48, 2, 32, [100, 45], 0, "ptd", "bf16"),  # 24 query heads on a key head
    ("bf16", 64, 40, 1, 128, [257, 9], 0, "ptd", "bf16"),
    ("e4m3", 64, 3, 1, 16, [1000, 15], 0, "ptd", "bf16"),
    ("bf16", 128, 7, 1, 16, [400, 100, 99, 3, 0, 1], 100, "ptd", "bf16"),
    ("f16", 64, 8, 4, 7, [50, 51, 52, 1, 2, 300], 1, "ptd", "f16"),
    ("e4m3", 128, 8, 2, 16, [600, 255, 256, 257], 256, "phtd", "bf16"),
    ("bf16", 128, 16, 4, 16, [5000, 1, 1, 1, 1, 1, 3000], 0, "ptd", "bf16"),
    ("f16", 128, 5, 1, 16, [20011], 0, "ptd", "bf16"),
    ("e4m3", 128, 6, 1, 64, [30001, 12], 0, "ptd", "bf16"),
    ("bf16", 64, 2, 2, 16, [int(x) for x in np.random.default_rng(0).integers(0, 90, 200)], 0, "ptd", "bf16"),
]


@pytest.mark.parametrize("kind,d,hq,hk,page,lens,window,order,out_t", ATTN)
def test_attention(kind, d, hq, hk, page, lens, window, order, out_t):
    tq = _tq()
    c = Case(len(lens) + d, kind, d, hq, hk, page, lens, order, junk=float("nan"))
    q = c.queries(7)
    ws = tq.workspace(tq.tq_attn_workspace(c.cache, c.m, hq))
    out = tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d, window, out_dtype=tq.TQ_BF16 if out_t == "bf16" else tq.TQ_F16,
                     ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    c.check_attn(q, out, d ** -0.5, window)
    assert (ws[:65536] == 0).all()  # the counters are left as they were found
    again = tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d, window, out=torch.empty_like(out), ws=ws)
    assert torch.equal(_bytes(out), _bytes(again))


@pytest.mark.parametrize("kind,d,hq,hk,lens", [
    ("e4m3", 128, 8, 8, [40000, 39001, 17, 0]),   # neighbouring heads of 128 bytes: pairs of warps
    ("e4m3", 64, 8, 8, [50001, 31999]),           # of 64 bytes: four warps
    ("f16", 64, 24, 1, [30011, 30000, 29000]),    # 24 query heads on one key head, two groups of them
    ("e4m3", 96, 10, 5, [33333, 33334, 33335]),   # an odd number of heads: no teams
    ("bf16", 256, 16, 2, [9000, 3]),
])
def test_attention_long_rows(kind, d, hq, hk, lens):
    """Enough keys that warps work in teams on neighbouring heads, and that rows are joined from many blocks."""
    tq = _tq()
    c = Case(d + len(lens), kind, d, hq, hk, 64, lens)
    q = c.queries(9)
    ws = tq.workspace(tq.tq_attn_workspace(c.cache, c.m, hq))
    out = tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d, ws=ws)
    c.check_attn(q, out, d ** -0.5)
    assert (ws[:65536] == 0).all()
    assert torch.equal(_bytes(out), _bytes(tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d, ws=ws)))


def test_attention_one_row_over_the_whole_gpu():
    """One key head: every block holds a part of the one item, joined in two rounds."""
    tq = _tq()
    for kind, d, hq in (("bf16", 128, 7), ("e4m3", 256, 16)):
        c = Case(2, kind, d, hq, 1, 128, [70001])
        q = c.queries(1)
        c.check_attn(q, tq.tq_attn(c.cache, q, c.pos_d, d ** -0.5, c.seq_d), d ** -0.5)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
def test_attention_sharp_and_flat_weights(kind):
    """Large scores of both signs (one key takes all, and keys whose weight underflows), zero and negative scales."""
    tq = _tq()
    c = Case(11, kind, 128, 8, 2, 16, [300, 17, 2, 1])
    q = c.queries(3) * 8
    for scale in (1.0, -1.0, 0.0, 2.0 ** -30):
        c.check_attn(q, tq.tq_attn(c.cache, q, c.pos_d, scale, c.seq_d), scale)


def test_attention_windows_ignore_what_is_before_them():
    """Keys before the window hold NaN, infinities and e4m3 NaN patterns."""
    tq = _tq()
    for kind in TYPES:
        c = Case(4, kind, 64, 4, 2, 16, [300, 64, 10], junk=float("nan"))
        q, w = c.queries(1), 37
        for i in range(c.m):
            for j in range(max(0, int(c.pos[i]) + 1 - w)):
                pg = int(c.table[c.seq[i], j // c.page])
                c.k[pg, j % c.page].copy_(torch.full((2, 64), float("nan")))
                c.v[pg, j % c.page].copy_(torch.full((2, 64), float("inf") if kind != "e4m3" else float("nan")))
        out = tq.tq_attn(c.cache, q, c.pos_d, 0.2, c.seq_d, w)
        c.check_attn(q, out, 0.2, w)


def test_attention_bad_pages_are_hidden():
    tq = _tq()
    c = Case(9, "bf16", 128, 8, 2, 16, [100, 100, 40, 16, 33])
    q = c.queries(5)
    table = c.cache.pages.clone()
    bad = [int(c.table[c.seq[0], 2]), int(c.table[c.seq[1], 6]), int(c.table[c.seq[3], 0])]
    for r, col, to in ((c.seq[0], 2, c.n_pages), (c.seq[1], 6, -1), (c.seq[3], 0, 2 ** 31 - 1)):
        table[int(r), col] = to
    cache = tq.KvCache(c.k, c.v, table)
    ws = tq.workspace(tq.tq_attn_workspace(cache, c.m, 8))
    out = tq.tq_attn(cache, q, c.pos_d, 0.1, c.seq_d, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
    c.check_attn(q, out, 0.1, hidden=bad)  # row 3 sees nothing: zeros
    # rows outside the table, and a position behind it
    seq = c.seq_d.clone()
    pos = c.pos_d.clone()
    seq[0], seq[1], pos[2] = -1, c.m, c.width * 16
    ws = tq.workspace(tq.tq_attn_workspace(cache, c.m, 8))
    out = tq.tq_attn(c.cache, q, pos, 0.1, seq, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
    assert (out[:3] == 0).all()
    c.pos[:3] = -1
    c.check_attn(q, out, 0.1)


def test_attention_rows_may_share_a_sequence():
    """Several new tokens of one request, each seeing what is before it."""
    tq = _tq()
    c = Case(8, "bf16", 128, 8, 2, 16, [70, 33])
    rows = [(0, 66), (0, 67), (0, 68), (0, 69), (1, 32), (1, 31)]
    c.seq = np.array([c.seq[r] for r, _ in rows], dtype=np.int32)
    c.pos = np.array([p for _, p in rows], dtype=np.int32)
    c.m = len(rows)
    q = c.queries(2)
    out = tq.tq_attn(c.cache, q, torch.from_numpy(c.pos).cuda(), 0.1, torch.from_numpy(c.seq).cuda())
    c.check_attn(q, out, 0.1)


def test_attention_many_rows():
    """The most rows a call takes; short rows beside one long one."""
    tq = _tq()
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 6, 4096)]
    lens[2000] = 3001
    c = Case(1, "f16", 64, 2, 1, 16, lens)
    q = c.queries(4)
    c.check_attn(q, tq.tq_attn(c.cache, q, c.pos_d, 0.125, c.seq_d), 0.125)


# ---- adapters -----------------------------------------------------------------------

LORA = [  # type, m, n, k, rank, adapters
    ("bf16", 1, 4096, 2560, 16, 4),
    ("f16", 1, 1, 512, 8, 1),
    ("bf16", 3, 1001, 512, 24, 2),
    ("f16", 8, 130, 1024, 64, 3),
    ("bf16", 17, 2048, 4096, 32, 5),
    ("f16", 64, 777, 1536, 128, 40),
    ("bf16", 100, 515, 512, 72, 100),
    ("f16", 333, 1024, 2048, 16, 7),
    ("bf16", 600, 384, 512, 8, 2),
    ("f16", 70, 96, 17408, 40, 1),
    ("bf16", 4096, 64, 512, 16, 33),
    ("f16", 257, 1000, 1024, 128, 3),
    ("bf16", 700, 515, 2560, 72, 9),
    ("bf16", 300, 129, 4608, 120, 300),
    ("f16", 512, 2561, 1536, 24, 1),
]


def _lora_inputs(kind, m, n, k, rank, na, seed=0):
    g = torch.Generator().manual_seed(seed + m + n)
    t = TYPES[kind]
    x = torch.randn((m, k), generator=g).to(t).cuda()
    a = (torch.randn((na, rank, k), generator=g) * k ** -0.5).to(t).cuda()
    b = torch.randn((na, n, rank), generator=g).to(t).cuda()
    s = (torch.rand(na, generator=g) * 2 + 0.1).cuda()
    ids = torch.randint(-1, na, (m,), generator=g).int()
    y = torch.randn((m, n), generator=g).cuda()
    return x, a, b, s, ids, y


def _check_lora(x, a, b, s, ids, y, out):
    want, bound = ref.lora(_num(x), _num(a), _num(b), np.ones(len(a)) if s is None else _num(s), ids.tolist(), _num(y))
    err = np.abs(_num(out) - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("kind,m,n,k,rank,na", LORA)
def test_lora(kind, m, n, k, rank, na):
    tq = _tq()
    x, a, b, s, ids, y = _lora_inputs(kind, m, n, k, rank, na)
    lora = tq.Lora(a, b, s)
    ws = tq.workspace(tq.tq_lora_workspace(lora, m))
    out = torch.full_like(y, float("nan"))
    tq.tq_lora(lora, x, ids.cuda(), y, out=out, ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    _check_lora(x, a, b, s, ids, y, out)
    assert (ws[:65536] == 0).all()
    again = y.clone()
    assert tq.tq_lora(lora, x, ids.cuda(), again, ws=ws) is again  # in place, the same bits
    assert torch.equal(out, again)
    # all tokens on one adapter, in runs and mixed, give each token the same bits
    one = torch.full_like(ids, na - 1)
    o1 = tq.tq_lora(lora, x, one.cuda(), y, out=torch.empty_like(y), ws=ws)
    _check_lora(x, a, b, s, one, y, o1)
    runs = torch.sort(ids).values
    o2 = tq.tq_lora(lora, x, runs.cuda(), y, out=torch.empty_like(y), ws=ws)
    _check_lora(x, a, b, s, runs, y, o2)


def test_lora_runs_shorter_than_a_tile():
    """Prompts of 17 tokens that take two adapters in turn stay in their order (more tiles than sorted tokens would
    make); single tokens of many adapters are sorted."""
    tq = _tq()
    x, a, b, s, ids, y = _lora_inputs("bf16", 600, 300, 512, 16, 2)
    for ids in (torch.arange(600).div(17, rounding_mode="floor").remainder(3).int() - 1, torch.arange(600).remainder(2).int()):
        _check_lora(x, a, b, s, ids, y, tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y)))


def test_lora_not_finite_tokens_stay_alone():
    """A token with an infinite or NaN input changes no other token, in small and large tiles."""
    tq = _tq()
    for kind, m in (("bf16", 20), ("f16", 300)):
        x, a, b, s, ids, y = _lora_inputs(kind, m, 200, 512, 16, 2)
        ids[:] = 1
        clean = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
        x[3, 7], x[m - 1, 100] = float("inf"), float("nan")
        dirty = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
        keep = [i for i in range(m) if i not in (3, m - 1)]
        assert torch.equal(clean[keep], dirty[keep])
        assert not torch.isfinite(dirty[3]).any() and dirty[m - 1].isnan().all()


def test_lora_columns_of_a_wider_output_and_no_scales():
    tq = _tq()
    for m, col, width in ((21, 0, 200), (21, 4, 200), (21, 3, 201), (21, 101, 203), (290, 3, 201)):
        x, a, b, _, ids, _ = _lora_inputs("bf16", m, 96, 512, 16, 3)
        wide = torch.randn((m, width)).cuda()
        keep = wide.clone()
        y = wide[:, col:col + 96]
        tq.tq_lora(tq.Lora(a, b), x, ids.cuda(), y)
        _check_lora(x, a, b, None, ids, keep[:, col:col + 96], y)
        keep[:, col:col + 96] = y
        assert torch.equal(keep, wide)


def test_lora_no_adapter_and_bad_index():
    tq = _tq()
    x, a, b, s, ids, y = _lora_inputs("f16", 12, 300, 512, 16, 3)
    lora = tq.Lora(a, b, s)
    ws = tq.workspace(tq.tq_lora_workspace(lora, 12))
    none = torch.full((12,), -1, dtype=torch.int32).cuda()
    assert torch.equal(tq.tq_lora(lora, x, none, y, out=torch.empty_like(y), ws=ws), y)
    none[3] = -2 ** 31
    assert torch.equal(tq.tq_lora(lora, x, none, y, out=torch.empty_like(y), ws=ws), y)
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    ids[5], ids[6] = 3, 2 ** 31 - 1
    out = tq.tq_lora(lora, x, ids.cuda(), y, out=torch.empty_like(y), ws=ws)
    assert tq.tq_workspace_status(ws) == tq.TQ_ERR_VALUE
    _check_lora(x, a, b, s, ids, y, out)


def test_lora_large_and_small_values():
    """A x outside fp16's range, and tiny: fp32 keeps both."""
    tq = _tq()
    for size in (300.0, 1e-4):
        x, a, b, s, ids, y = _lora_inputs("f16", 40, 64, 512, 16, 2)
        x, a = (x.float() * size).half(), (a.float() * 20 * (size if size > 1 else 1)).half()
        out = tq.tq_lora(tq.Lora(a, b, s), x, ids.cuda(), y, out=torch.empty_like(y))
        _check_lora(x, a, b, s, ids, y, out)


# ---- use -----------------------------------------------------------------------

def test_graphs_that_share_a_workspace_and_other_streams():
    """An append and attention step, and an adapter step, captured in two graphs on one workspace and replayed in turn
    with new positions and adapters; then the same calls on a stream of their own."""
    tq = _tq()
    c = Case(3, "bf16", 128, 8, 2, 16, [200, 33, 1])
    lx, la, lb, ls, lids, ly = _lora_inputs("bf16", 20, 300, 1024, 16, 4)
    lora, ids = tq.Lora(la, lb, ls), lids.cuda()
    px, _, _, _, pids, py = _lora_inputs("bf16", 320, 300, 1024, 16, 4)
    pids_d, po = pids.cuda(), torch.empty_like(py)
    ws = tq.workspace(max(tq.tq_attn_workspace(c.cache, 3, 8), tq.tq_lora_workspace(lora, 320)))
    qkv = torch.randn((3, 12 * 128)).cuda()
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    q, out = torch.empty((3, 8, 128), dtype=torch.bfloat16).cuda(), torch.empty((3, 8, 128), dtype=torch.bfloat16).cuda()
    lo = torch.empty_like(ly)

    def step():
        tq.tq_kv_append(c.cache, qkv, 8, c.pos_d, freq, seq=c.seq_d, q_out=q, ws=ws)
        tq.tq_attn(c.cache, q, c.pos_d, 0.1, c.seq_d, out=out, ws=ws)

    def adapt():
        tq.tq_lora(lora, lx, ids, ly, out=lo, ws=ws)
        tq.tq_lora(lora, px, pids_d, py, out=po, ws=ws)

    step()
    adapt()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step()
    with torch.cuda.graph(g2):
        adapt()
    for shift in (0, 1, 2):
        pos = c.pos - shift
        c.pos_d.copy_(torch.from_numpy(pos))
        ids.copy_((lids + 1 + shift) % 5 - 1)
        pids_d.copy_((pids + 1 + shift) % 5 - 1)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        saved = c.pos
        c.pos = pos
        c.check_attn(q, out, 0.1)
        c.pos = saved
        _check_lora(lx, la, lb, ls, ids.cpu(), ly, lo)
        _check_lora(px, la, lb, ls, pids_d.cpu(), py, po)
    c.pos_d.copy_(torch.from_numpy(c.pos))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q2 = tq.tq_kv_append(c.cache, qkv, 8, c.pos_d, freq, seq=c.seq_d, stream=s)
    o2 = tq.tq_attn(c.cache, q2, c.pos_d, 0.1, c.seq_d, stream=s)
    l2 = tq.tq_lora(lora, lx, ids, ly, out=torch.empty_like(ly), stream=s)
    s.synchronize()
    c.check_attn(q2, o2, 0.1)
    _check_lora(lx, la, lb, ls, ids.cpu(), ly, l2)


def test_adapters_between_projections():
    """Projection, adapters, projection, adapters, launched without a pause and replayed from a graph: the projections'
    and the prompt adapters' kernels share tensor memory and overlap their launches.  Each output is checked from the
    inputs of its own call."""
    import tqsynth
    tq = _tq()
    m, n, k = 300, 1536, 1024
    cb = tqsynth.codebook(1)
    hw = tqsynth.Weight(1, 0, 0, n, k, cb)
    w = tq.DeviceWeight.from_host(hw.codes, hw.scales, torch.from_numpy(cb.view(np.int16)).cuda(), n, k)
    x, a, b, s, ids, _ = _lora_inputs("f16", m, n, k, 16, 5)
    lora, ids_d = tq.Lora(a, b, s), ids.cuda()
    ys = [torch.empty((m, n)).cuda() for _ in range(6)]
    outs = [torch.empty((m, n)).cuda() for _ in range(6)]
    ws = tq.workspace(max(tq.tq_gemm_workspace(n, k, m), tq.tq_lora_workspace(lora, m)))

    def chain():
        for y, o in zip(ys, outs):
            tq.tq_gemm(w, x, y, ws)
            tq.tq_lora(lora, x, ids_d, y, out=o, ws=ws)

    chain()
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    first = outs[0].clone()
    _check_lora(x, a, b, s, ids, ys[0], first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for t in ys + outs:
        t.zero_()
    g.replay()
    g.replay()
    assert tq.tq_workspace_status(ws) == tq.TQ_OK
    assert all(torch.equal(y, ys[0]) for y in ys) and all(torch.equal(o, first) for o in outs)


def test_empty_calls():
    tq = _tq()
    c = Case(3, "f16", 64, 4, 2, 16, [5])
    none = torch.empty(0, dtype=torch.int32).cuda()
    assert tq.tq_kv_append(c.cache, torch.empty((0, 8 * 64)).cuda(), 4, none).shape == (0, 4, 64)
    assert tq.tq_attn(c.cache, torch.empty((0, 4, 64), dtype=torch.float16).cuda(), none, 1.0).shape == (0, 4, 64)
    x, a, b, s, _, _ = _lora_inputs("f16", 1, 300, 512, 16, 3)
    assert tq.tq_lora(tq.Lora(a, b, s), x[:0], none, torch.empty((0, 300)).cuda()).shape == (0, 300)


# ---- the stack with its attention -----------------------------------------------------

@pytest.mark.parametrize("m,kind,adapters", [(1, "bf16", False), (3, "e4m3", True), (40, "f16", True)])
def test_attention_stack(m, kind, adapters):
    """Two layers, three steps of decoding, stage by stage against the oracle: each stage is checked from the GPU's own
    input to it."""
    import oracle
    import tqsynth
    from decode_matmul_b200.attention import AttentionStack
    from gpu_util import TOL
    tq = _tq()
    shape = tqsynth.StackShape("attn-test", 2, 512, 1024, 256, 1536)
    cb = tqsynth.codebook(3)
    cbd = torch.from_numpy(cb.view(np.int16)).cuda()
    host = [{op: tqsynth.Weight(3, l, i, n, k, cb) for i, (op, n, k) in enumerate(shape.ops())} for l in range(2)]
    layers = [{op: tq.DeviceWeight.from_host(w.codes, w.scales, cbd, w.n, w.k) for op, w in L.items()} for L in host]
    rng = np.random.default_rng(m)
    lens = [int(x) for x in rng.integers(1, 60, m)]
    cs = [Case(20 + l, kind, 128, 8, 2, 16, [n + 3 for n in lens], shuffle_seq=False) for l in range(2)]
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    loras = None
    if adapters:
        loras = [{op: tq.Lora(*_lora_inputs("bf16", 1, shape.q_dim if op == "q" else shape.kv_dim, 512, 16, 3, seed=l)[1:4])
                  for op in ("q", "v")} for l in range(2)]
    stack = AttentionStack(layers, [c.cache for c in cs], freq, adapters=loras)
    ids = torch.from_numpy(rng.integers(-1, 3, m).astype(np.int32)).cuda()
    h = torch.from_numpy(tqsynth.activations(1, m, 512).view(np.int16)).cuda()
    for step in range(3):
        pos = np.array([n + step for n in lens], dtype=np.int32)
        if m > 1:
            pos[1] = -1  # a padded row
        pos_d = torch.from_numpy(pos).cuda()
        before = [_bytes(cs[1].k), _bytes(cs[1].v)]
        out = stack.forward(h, pos_d, 5, adapter=ids if adapters else None)
        b = stack.buffers(m)
        assert tq.tq_workspace_status(b["ws"]) == tq.TQ_OK
        # the last layer's stages from the GPU's own inputs
        x = b["hand"][3].cpu().numpy().view(np.uint16)
        W = {op: (w.codes, w.scales, w.codebook, w.n, w.k) for op, w in host[1].items()}
        ys, _ = oracle.stack_phase(0, x, m, {op: W[op] for op in "qkv"}, oracle.stack_phase_seed(5, 1, 0))
        y = np.concatenate([ys[op] for op in "qkv"], axis=1)
        if adapters:
            xb = tqsynth.bf16_to_f64(x).reshape(m, -1)
            for op, col in (("q", 0), ("v", 1280)):
                L = loras[1][op]
                y[:, col:col + L.n] = ref.lora(xb, _num(L.a), _num(L.b), _num(L.scale), ids.tolist(), y[:, col:col + L.n])[0]
        assert oracle.rel_err(_num(b["y"]), y) < TOL
        c = cs[1]
        c.pos = pos
        _check_append(c, b["y"], b["q"], before, freq, False)
        c.check_attn(b["q"], b["attn"], 128 ** -0.5)
        a = b["attn"].view(torch.int16).cpu().numpy().view(np.uint16).reshape(m, -1)
        _, hand = oracle.stack_phase(1, a, m, {"o": W["o"]}, oracle.stack_phase_seed(5, 1, 1))
        got = tqsynth.bf16_to_f64(b["hand"][1].cpu().numpy().view(np.uint16))
        want = tqsynth.bf16_to_f64(hand)
        # one bf16 step, and the linear layers' bound on its input
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -7 + 2 * TOL * np.maximum(np.abs(want), np.sqrt((want ** 2).mean()))).all()
        x2 = b["hand"][2].cpu().numpy().view(np.uint16)
        _, hand = oracle.stack_phase(3, x2, m, {"down": W["down"]}, oracle.stack_phase_seed(5, 1, 3))
        got, want = tqsynth.bf16_to_f64(out.cpu().numpy().view(np.uint16)), tqsynth.bf16_to_f64(hand)
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -7 + 2 * TOL * np.maximum(np.abs(want), np.sqrt((want ** 2).mean()))).all()
        h = out
    # a captured step gives the bits of an eager one (the same tokens again: the cache slots are rewritten)
    h0, o0 = h.clone(), torch.empty_like(h)
    eager = stack.forward(h0, pos_d, 5, adapter=ids if adapters else None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stack.forward(h0, pos_d, 5, adapter=ids if adapters else None, out=o0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, o0)
