"""Three operators of a decode step around the trellis-coded linear layers:

  append   rotate the queries and keys of new tokens by their position and
           append keys and values to a paged cache (``tq_kv_append``)
  attn     attention of one new token per row over the paged cache
           (``tq_attn``)
  lora     low-rank adapters of many requests beside a shared projection
           (``tq_lora``)

``run`` computes them in plain torch where ``own`` is false and calls the
library where it is true.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "e4m3": 1}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one user's next token enters the cache: latency only (32 query heads on 8 key heads of 128)
        dict(name="append-1", op="append", m=1, q_heads=32, kv_heads=8, head_dim=128, page=16, type="bf16",
             rot=128, interleaved=False, theta=1e6, far=40960, prompt=False, pad=0, rng=1),
        # a decode batch of 64 requests far into their contexts, 8-bit cache, three padded rows
        dict(name="append-64-e4m3", op="append", m=64, q_heads=48, kv_heads=8, head_dim=128, page=16, type="e4m3",
             rot=64, interleaved=False, theta=1e7, far=131072, prompt=False, pad=3, rng=2),
        # one prompt of 4001 tokens: bandwidth
        dict(name="append-prompt-4001", op="append", m=4001, q_heads=32, kv_heads=8, head_dim=128, page=32, type="f16",
             rot=128, interleaved=True, theta=5e5, far=131072, prompt=True, pad=0, rng=3),
        # one user, a short chat: latency and the split over the length
        dict(name="attn-1", op="attn", m=1, q_heads=32, kv_heads=8, head_dim=128, page=16, type="bf16",
             longest=777, shortest=777, window=0, pad=0, rng=4),
        # 64 requests of very different lengths
        dict(name="attn-64-ragged", op="attn", m=64, q_heads=32, kv_heads=8, head_dim=128, page=16, type="bf16",
             longest=8192, shortest=3, window=0, pad=0, rng=5),
        # few users with long documents, 8-bit cache
        dict(name="attn-16-long-e4m3", op="attn", m=16, q_heads=48, kv_heads=8, head_dim=128, page=64, type="e4m3",
             longest=65536, shortest=20000, window=0, pad=0, rng=6),
        # narrow heads in odd groups, odd pages, a sliding window and padded rows
        dict(name="attn-33-window", op="attn", m=33, q_heads=20, kv_heads=4, head_dim=64, page=24, type="f16",
             longest=16000, shortest=1, window=4096, pad=2, rng=7),
        # wide heads that share one key head
        dict(name="attn-24-wide", op="attn", m=24, q_heads=8, kv_heads=1, head_dim=256, page=16, type="bf16",
             longest=32768, shortest=1000, window=0, pad=0, rng=8),
        # one user with one adapter beside the query projection: latency
        dict(name="lora-1", op="lora", m=1, n=4096, k=2560, rank=16, adapters=4, type="bf16", runs=False, none=0, rng=9),
        # a decode batch whose 64 requests use 24 adapters in any order, some none, beside the down projection
        dict(name="lora-64", op="lora", m=64, n=5120, k=17408, rank=32, adapters=24, type="f16", runs=False, none=5,
             rng=10),
        # prompts of eleven requests in one batch beside gate and up
        dict(name="lora-prompts-1000", op="lora", m=1000, n=19456, k=2560, rank=64, adapters=11, type="bf16", runs=True,
             none=0, rng=11),
        # the largest batch beside a down projection
        dict(name="lora-prompts-4096", op="lora", m=4096, n=4096, k=14336, rank=16, adapters=40, type="bf16", runs=True,
             none=300, rng=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "lora", "lora"])
    if op == "lora":
        m = _log(rng, 1, 4096)
        n = rng.choice([1024, 2560, 4096, 5120, 6144, 14336, 19456, 1 + _log(rng, 100, 9000)])
        k = 512 * _log(rng, 1, 34)
        while m * n > 20_000_000 or m * k > 60_000_000:
            m = max(1, m // 2)
        none = rng.randint(0, m // 4)
        return dict(op=op, m=m, n=n, k=k, rank=8 * rng.choice([1, 2, 2, 4, 8, 16, rng.randint(1, 16)]),
                    adapters=_log(rng, 1, 48), type=rng.choice(["bf16", "f16"]), runs=rng.random() < 0.5, none=none,
                    rng=rng.randrange(1 << 30))
    head_dim = rng.choice([64, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    while q_heads * head_dim > 8192:
        q_heads -= kv_heads
    kind = rng.choice(["bf16", "f16", "e4m3"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128])
    if op == "append":
        prompt = rng.random() < 0.4
        m = _log(rng, 1, 4000) if prompt else _log(rng, 1, 256)
        while m * (q_heads + 2 * kv_heads) * head_dim > 24_000_000:
            m = max(1, m // 2)
        rot = rng.choice([head_dim, head_dim, head_dim // 2])
        return dict(op=op, m=m, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, type=kind, rot=rot,
                    interleaved=rng.random() < 0.4, theta=rng.choice([1e4, 5e5, 1e6, 1e7]), far=_log(rng, 4100, 1_000_000),
                    prompt=prompt, pad=0 if m == 1 else rng.randint(0, m // 8), rng=rng.randrange(1 << 30))
    m = _log(rng, 1, 256)
    longest = _log(rng, 1, 65536)
    while m * longest * kv_heads * head_dim > 300_000_000:
        longest = max(1, longest // 2)
    shortest = rng.choice([1, longest, max(1, longest // 4)])
    window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    return dict(op=op, m=m, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, type=kind, longest=longest,
                shortest=shortest, window=window, pad=0 if m == 1 else rng.randint(0, m // 8),
                rng=rng.randrange(1 << 30))


def _positions(case):
    """Positions of the new tokens (host side, fixed by the case; -1 = a padded row)."""
    r = random.Random(case["rng"])
    m = case["m"]
    if case["op"] == "append":
        if case["prompt"]:
            first = r.randrange(0, case["far"] - m)
            pos = list(range(first, first + m))
        else:
            pos = [r.randrange(0, case["far"]) for _ in range(m)]
            pos[0] = case["far"] - 1
    else:
        lens = [_log(r, case["shortest"], case["longest"]) for _ in range(m)]
        lens[r.randrange(m - case["pad"])] = case["longest"]
        pos = [n - 1 for n in lens]
    return pos[:m - case["pad"]] + [-1] * case["pad"]


def _slots(case):
    """Block-table row of each token: one request for a prompt, else a slot of its own in any order."""
    if case.get("prompt"):
        return [0] * case["m"]
    slots = list(range(case["m"]))
    random.Random(case["rng"] + 2).shuffle(slots)
    return slots


def _adapters(case):
    """Adapter of each token (host side, fixed by the case; -1 = none)."""
    r = random.Random(case["rng"])
    m, used = case["m"], case["m"] - case["none"]
    ids = [i % case["adapters"] for i in range(used)]
    ids = sorted(ids) + [-1] * case["none"]
    if not case["runs"]:
        r.shuffle(ids)
    return ids


def _seen(case):
    """Keys each row of an attention case sees."""
    w = case["window"]
    return [min(p + 1, w) if w else p + 1 for p in _positions(case)]


def work(case):
    m = case["m"]
    if case["op"] == "lora":
        used = len(set(a for a in _adapters(case) if a >= 0))
        tokens = m - case["none"]
        n, k, r = case["n"], case["k"], case["rank"]
        return dict(bytes=used * (r * k + n * r) * 2 + tokens * k * 2 + m * n * 8 + m * 4, flops=2 * tokens * r * (k + n) + m * n)
    hq, hk, d, e = case["q_heads"], case["kv_heads"], case["head_dim"], BYTES[case["type"]]
    if case["op"] == "append":
        live = sum(p >= 0 for p in _positions(case))
        return dict(bytes=live * (hq + 2 * hk) * d * 4 + m * hq * d * 2 + live * 2 * hk * d * e + m * 8,
                    flops=3 * live * (hq + hk) * case["rot"])
    keys = sum(_seen(case))
    return dict(bytes=keys * hk * d * 2 * e + m * hq * d * 4 + m * 8, flops=4 * keys * hq * d)


# ---- inputs ------------------------------------------------------------------

def _to_e4m3(x):
    """Nearest e4m3 value (ties to even, saturating at 448) of a float64 tensor, as float64."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.frexp(a).exponent.to(torch.float64).sub(1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x).clamp(-448.0, 448.0)


def _pages(case, pos, slots):
    """A block table in random page order.  An attention case has a page for every key; an append case
    only for the pages that are written (the older entries point at page 0, which nothing writes)."""
    ps, m = case["page"], case["m"]
    width = max(pos) // ps + 1
    table = np.zeros((1 if case.get("prompt") else m, width), dtype=np.int64)
    spots = []
    for i, p in enumerate(pos):
        if p >= 0:
            first = p // ps if case["op"] == "append" else 0
            spots += [(slots[i], j) for j in range(first, p // ps + 1)]
    spots = sorted(set(spots))
    ids = np.arange(1, len(spots) + 1)
    np.random.default_rng(case["rng"]).shuffle(ids)
    if spots:
        at = np.asarray(spots)
        table[at[:, 0], at[:, 1]] = ids
    return torch.from_numpy(table.astype(np.int32)).cuda(), len(spots) + 2


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + case["rng"] % 1000003)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        return out.normal_(0.0, scale, generator=gen)

    s = dict(case=case)
    m = case["m"]
    if case["op"] == "lora":
        t = TYPES[case["type"]]
        n, k, r, na = case["n"], case["k"], case["rank"], case["adapters"]
        s["x"] = normal(m, k, dtype=t)
        s["a"] = normal(na, r, k, dtype=t, scale=k ** -0.5)
        s["b"] = normal(na, n, r, dtype=t, scale=0.3)
        s["s"] = torch.empty(na, device="cuda").uniform_(0.25, 2.0, generator=gen)
        s["y"] = normal(m, n)
        s["ids"] = torch.tensor(_adapters(case), dtype=torch.int32, device="cuda")
        if own:
            import decode_matmul_b200 as tq
            s["out"] = torch.empty_like(s["y"])
            s["lora"] = tq.Lora(s["a"], s["b"], s["s"])
            s["ws"] = tq.workspace(tq.tq_lora_workspace(s["lora"], m))
        return s
    hq, hk, d, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    pos, slots = _positions(case), _slots(case)
    s["pages"], n_pages = _pages(case, pos, slots)
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["seq"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
    s["rows"] = torch.tensor([i for i, p in enumerate(pos) if p >= 0], dtype=torch.int64, device="cuda")
    e4m3 = case["type"] == "e4m3"
    s["ks"] = torch.empty(hk, device="cuda").uniform_(0.005, 0.02, generator=gen) if e4m3 else None
    s["vs"] = torch.empty(hk, device="cuda").uniform_(0.005, 0.02, generator=gen) if e4m3 else None
    for name in ("kc", "vc"):
        c = normal(n_pages, ps, hk, d, dtype=torch.float16 if e4m3 else TYPES[case["type"]])
        # an 8-bit cache holds values around +-100, which times its scales are around one
        s[name] = (c * 80).clamp(-448, 448).to(torch.float8_e4m3fn) if e4m3 else c
    if case["op"] == "append":
        s["qkv"] = normal(m, (hq + 2 * hk) * d)
        half = case["rot"] // 2
        s["freq"] = case["theta"] ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    else:
        s["q"] = normal(m, hq, d, dtype=torch.bfloat16 if case["type"] == "bf16" else torch.float16)
        s["scale"] = d ** -0.5
    if own:
        import decode_matmul_b200 as tq
        s["cache"] = tq.KvCache(s["kc"], s["vc"], s["pages"], s["ks"], s["vs"])
        if case["op"] == "append":
            s["ws"] = tq.workspace(tq.tq_kv_append_workspace())
            s["out"] = torch.empty((m, hq, d), dtype=torch.bfloat16 if case["type"] == "bf16" else torch.float16,
                                   device="cuda")
        else:
            s["ws"] = tq.workspace(tq.tq_attn_workspace(s["cache"], m, hq))
            s["out"] = torch.empty((m, hq, d), dtype=torch.bfloat16, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def _values(cache, scale):
    """What a cache stands for: 16-bit caches as they are, 8-bit ones times their scales."""
    return cache if scale is None else cache.float() * scale[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    """x [m][heads][d]; cos, sin [m][1][rot/2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _append(s):
    c = s["case"]
    hq, hk, d, ps, m = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], c["m"]
    e4m3 = c["type"] == "e4m3"
    # an 8-bit value next to a rounding border needs more than 32 bits; the angles of far positions always do
    t = torch.float64 if e4m3 else torch.float32
    rows = s["rows"]
    pos = s["pos"][rows].long()
    angle = (pos.double()[:, None] * s["freq"])[:, None, :]
    cos, sin = torch.cos(angle).to(t), torch.sin(angle).to(t)
    x = s["qkv"][rows].view(-1, hq + 2 * hk, d)
    qt = torch.bfloat16 if c["type"] == "bf16" else torch.float16
    q = torch.zeros((m, hq, d), dtype=qt, device=x.device)
    q[rows] = _rotate(x[:, :hq].float(), cos.float(), sin.float(), c["rot"], c["interleaved"]).to(qt)
    k = _rotate(x[:, hq:hq + hk].to(t), cos, sin, c["rot"], c["interleaved"])
    v = x[:, hq + hk:].to(t)
    page = s["pages"][s["seq"][rows].long(), pos // ps].long()
    for cache, new, scale in ((s["kc"], k, s["ks"]), (s["vc"], v, s["vs"])):
        if e4m3:
            new = _to_e4m3(new / scale.double()[:, None]).float().to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[page, pos % ps] = new.view(torch.uint8)
        else:
            cache[page, pos % ps] = new.to(cache.dtype)
    return [q, _values(s["kc"], s["ks"]), _values(s["vc"], s["vs"])]


def _attn(s):
    c = s["case"]
    hq, hk, d, ps, m, w = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], c["m"], c["window"]
    out = torch.empty((m, hq, d), dtype=torch.bfloat16, device="cuda")
    longest = c["longest"]
    chunk = max(1, (1 << 29) // (longest * hk * d))
    j = torch.arange(longest, device="cuda")
    for i in range(0, m, chunk):
        pos = s["pos"][i:i + chunk].long()[:, None]
        page = s["pages"][s["seq"][i:i + chunk].long()][:, j // ps].long()
        seen = j <= pos
        if w:
            seen &= j > pos - w
        kc, vc = (x.view(torch.uint8)[page, j % ps].view(x.dtype) if x.element_size() == 1 else x[page, j % ps]
                  for x in (s["kc"], s["vc"]))
        kc, vc = _values(kc, s["ks"]).float(), _values(vc, s["vs"]).float()
        q = s["q"][i:i + chunk].float().view(-1, hk, hq // hk, d)
        score = torch.einsum("mhgd,mjhd->mhgj", q, kc) * s["scale"]
        seen = seen[:, None, None, :]
        score = torch.where(seen, score, -3e38)
        p = torch.where(seen, torch.exp(score - score.amax(-1, keepdim=True)), 0.0)
        o = torch.einsum("mhgj,mjhd->mhgd", p, vc) / p.sum(-1, keepdim=True).clamp(min=1e-30)
        out[i:i + chunk] = o.reshape(-1, hq, d).to(torch.bfloat16)
    return out


def _lora(s):
    a, b = s["a"].float(), s["b"].float()
    na, r, k = a.shape
    h = (s["x"].float() @ a.view(na * r, k).t()).view(-1, na, r)
    mine = s["ids"][:, None] == torch.arange(na, device="cuda")
    h = torch.where(mine[:, :, None], h * s["s"][:, None], 0.0)
    return s["y"] + h.view(-1, na * r) @ b.transpose(1, 2).reshape(na * r, -1)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "attn": _attn, "lora": _lora}[op](s)
    import decode_matmul_b200 as tq
    c = s["case"]
    if op == "append":
        tq.tq_kv_append(s["cache"], s["qkv"], c["q_heads"], s["pos"], s["freq"], interleaved=c["interleaved"],
                        seq=s["seq"], q_out=s["out"], ws=s["ws"])
        return [s["out"], _values(s["kc"], s["ks"]), _values(s["vc"], s["vs"])]
    if op == "attn":
        return tq.tq_attn(s["cache"], s["q"], s["pos"], s["scale"], seq=s["seq"], window=c["window"], out=s["out"],
                          ws=s["ws"])
    return tq.tq_lora(s["lora"], s["x"], s["ids"], s["y"], out=s["out"], ws=s["ws"])


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    m = case["m"]
    if case["op"] == "lora":
        want = s["y"].double()
        ids = _adapters(case)
        for a in sorted(set(ids) - {-1}):
            t = torch.tensor([i for i, x in enumerate(ids) if x == a], device="cuda")
            h = torch.matmul(s["x"][t].double(), s["a"][a].double().T)
            want[t] += s["s"][a].double() * torch.matmul(h, s["b"][a].double().T)
        return want
    hq, hk, d, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    pos, table, seq = _positions(case), s["pages"].long(), _slots(case)
    if case["op"] == "attn":
        want = torch.zeros((m, hq, d), dtype=torch.float64, device="cuda")
        for i, p in enumerate(pos):
            first = max(0, p + 1 - case["window"]) if case["window"] else 0
            if p < 0:
                continue
            at = torch.arange(first, p + 1, device="cuda")
            where = table[seq[i], torch.div(at, ps, rounding_mode="floor")]
            for h in range(hk):
                ks = 1.0 if s["ks"] is None else s["ks"][h].double()
                vs = 1.0 if s["vs"] is None else s["vs"][h].double()
                kk = s["kc"][:, :, h].view(torch.uint8)[where, at % ps].view(s["kc"].dtype).double() * ks
                vv = s["vc"][:, :, h].view(torch.uint8)[where, at % ps].view(s["vc"].dtype).double() * vs
                q = s["q"][i, h * (hq // hk):(h + 1) * (hq // hk)].double()
                want[i, h * (hq // hk):(h + 1) * (hq // hk)] = torch.softmax((q @ kk.T) * s["scale"], dim=1) @ vv
        return want
    rot, half = case["rot"], case["rot"] // 2
    idx = torch.arange(half, device="cuda")
    lo, hi = (2 * idx, 2 * idx + 1) if case["interleaved"] else (idx, idx + half)
    x = s["qkv"].double().view(m, hq + 2 * hk, d)
    live = torch.tensor([p >= 0 for p in pos], device="cuda")
    z = torch.polar(torch.ones((m, 1, half), dtype=torch.float64, device="cuda"),
                    s["pos"].double()[:, None, None] * s["freq"])
    turned = x[:, :hq + hk].clone()
    pair = torch.complex(turned[..., lo], turned[..., hi]) * z
    turned[..., lo], turned[..., hi] = pair.real, pair.imag
    q = torch.where(live[:, None, None], turned[:, :hq], 0.0)
    caches = []
    for cache, new, scale in ((s["kc"], turned[:, hq:], s["ks"]), (s["vc"], x[:, hq + hk:], s["vs"])):
        want = cache.double()
        if scale is not None:
            levels = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
            levels = torch.unique(levels[torch.isfinite(levels)])
            ratio = (new / scale.double()[:, None]).clamp(-448.0, 448.0).contiguous()
            up = torch.searchsorted(levels, ratio).clamp(max=len(levels) - 1)
            down = (up - 1).clamp(min=0)
            low, high = levels[down], levels[up]
            nearer = torch.where(ratio - low < high - ratio, low, high)
            # halfway: the neighbour with the even last bit, which is the one that halving the step keeps
            even = torch.where(_even(low), low, high)
            new = torch.where(ratio - low == high - ratio, even, nearer)
        for i, p in enumerate(pos):
            if p >= 0:
                want[table[seq[i], p // ps], p % ps] = new[i]
        caches.append(want if scale is None else want * scale.double()[:, None])
    return [q] + caches


def _even(level):
    """Whether the e4m3 pattern of these values ends in a zero bit."""
    return (level.float().to(torch.float8_e4m3fn).view(torch.uint8) & 1) == 0
