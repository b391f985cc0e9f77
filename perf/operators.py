"""Measured cases of the paged-cache operators: attention of new tokens over a
paged key/value cache, rotary positions (on tensors, and fused with the append
to the cache), and the page operations (taking rows over, growing, freeing,
compacting).

``run`` computes each operator either with the library (``own`` true) or in
its plain form: elementary torch operations in 32 bits (angles in 64), rounded
once at the end. ``exact`` is the definition again, in 64 bits, one sequence
and one head group at a time.

Conventions: sequence b of a batch has T_b new tokens, rows cu[b] .. cu[b+1]
of the packed tensors, and L_b cached tokens in all, the new ones included;
its new token i sits at position L_b - T_b + i. Position t of sequence b lies
in page table[b, t // page], row t % page.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _lib():
    import exact_tiled_attention_38_b200 as eta

    return eta


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # Attention over the cache.
        # A small interactive batch, one token each: the latency of a call counts.
        dict(name="attend_decode_small", op="attend", dtype="bf16", B=4, Hq=32, Hkv=8, d=128, page=16,
             tmin=1, tmax=1, lmin=30, lmax=700, window=0, lens=1),
        # The ragged decode batch of the benchmark (64 sequences of 1K-8K), paged.
        dict(name="attend_decode_ragged", op="attend", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, page=64,
             tmin=1, tmax=1, lmin=1024, lmax=8192, window=0, lens=2),
        # A mixed serving batch: single tokens and chunks together, a sliding
        # window, the smaller head size, small pages, odd lengths.
        dict(name="attend_mixed_window", op="attend", dtype="f16", B=9, Hq=16, Hkv=2, d=64, page=16,
             tmin=1, tmax=301, lmin=301, lmax=16001, window=4096, lens=3),
        # One chunk of a long prompt over what is cached of it already.
        dict(name="attend_chunk_long", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, page=128,
             tmin=1024, tmax=1024, lmin=65536, lmax=65536, window=0, lens=4),
        # Rotary positions.
        # q and k of a training step (the causal 2K workload's sizes).
        dict(name="rope_forward_2k", op="rope", dtype="bf16", B=4, Hq=16, Hkv=16, N=2048, d=128, rot=128,
             interleaved=False, scaling="none", first=0, grad=False),
        # Their gradients in a long-context step: far positions, scaled by
        # parts, a rotated quarter of the head, neighbouring pairs.
        dict(name="rope_gradient_32k", op="rope", dtype="f16", B=1, Hq=32, Hkv=8, N=32768, d=64, rot=32,
             interleaved=True, scaling="parts", first=98304, grad=True),
        # One decode step's q, k, v: rotated, and k, v put into the cache.
        dict(name="append_decode", op="append", dtype="bf16", B=64, Hq=32, Hkv=8, d=128, rot=128, page=64,
             interleaved=False, scaling="none", tmin=1, tmax=1, lmin=1024, lmax=8192, lens=5),
        # The same for ragged prompt chunks.
        dict(name="append_chunks", op="append", dtype="bf16", B=9, Hq=32, Hkv=8, d=128, rot=64, page=16,
             interleaved=True, scaling="bands", tmin=200, tmax=1801, lmin=1801, lmax=9000, lens=6),
        # Page operations.
        # One step of a serving batch: a few rows end, a few start, the rest grow by a token.
        dict(name="update_step", op="update", dtype="bf16", layers=2, B=64, Hkv=8, d=128, page=16, lmin=100, lmax=1000,
             take="serve", lens=7),
        # A beam step: rows take over other rows; all layers' last pages are copied.
        dict(name="update_beams", op="update", dtype="bf16", layers=16, B=96, Hkv=8, d=128, page=64, lmin=200, lmax=600,
             take="beams", lens=8),
        # Compaction of a small cache, and of a large one.
        dict(name="compact_small", op="compact", dtype="f16", layers=1, B=7, Hkv=2, d=64, page=16, lmin=1, lmax=300,
             moves=20, spare=150, lens=9),
        dict(name="compact_large", op="compact", dtype="bf16", layers=8, B=64, Hkv=8, d=128, page=32, lmin=100, lmax=2000,
             moves=700, spare=1000, lens=10),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "append", "update", "compact"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), lens=rng.randrange(1 << 20))
    Hkv = _spread(rng, 1, 8)
    d = rng.choice([64, 64, 128, 128, 128, 32, 80, 96])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "attend":
        G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
        kind = rng.choice(["decode", "few", "chunk"])
        tmax = 1 if kind == "decode" else _spread(rng, 2, 8) if kind == "few" else _spread(rng, 9, 900)
        lmax = _spread(rng, max(tmax, 20), 30000)
        most = min(3e8 / (Hkv * G * tmax * lmax), 3e8 / (lmax * Hkv * d))  # scores; values of the cache
        B = _spread(rng, 1, max(1, min(96, int(most))))
        c.update(B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, tmin=rng.choice([1, tmax]), tmax=tmax,
                 lmin=rng.randrange(tmax, lmax + 1), lmax=lmax,
                 window=rng.choice([0, 0, _spread(rng, 1, lmax)]))
    elif op == "rope":
        G = rng.choice([1, 2, 3, 4, 8])
        N = _spread(rng, 1, 16384)
        B = _spread(rng, 1, max(1, min(16, int(8e7 / (N * Hkv * (G + 1) * d)))))
        c.update(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "base", "parts", "bands"]), first=_spread(rng, 1, 1 << 20),
                 grad=rng.random() < 0.5)
    elif op == "append":
        G = rng.choice([1, 2, 3, 4, 8])
        tmax = rng.choice([1, _spread(rng, 1, 1500)])
        lmax = _spread(rng, max(tmax, 20), 8000)
        B = _spread(rng, 1, max(1, min(96, int(8e7 / (tmax * Hkv * (G + 2) * d)), int(2e8 / (lmax * Hkv * d)))))
        c.update(B=B, Hq=Hkv * G, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]), page=page,
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "parts", "bands"]),
                 tmin=rng.choice([1, tmax]), tmax=tmax, lmin=rng.randrange(tmax, lmax + 1), lmax=lmax)
    else:
        layers = _spread(rng, 1, 8)
        lmax = _spread(rng, 20, 2000)
        B = _spread(rng, 2, max(2, min(128, int(1.5e8 / (layers * lmax * Hkv * d)))))
        c.update(layers=layers, B=B, Hkv=Hkv, d=d, page=page, lmin=rng.randrange(1, lmax + 1), lmax=lmax)
        if op == "update":
            c.update(take=rng.choice(["serve", "beams"]))
        else:
            held = _pages_of(c)
            c.update(moves=rng.randrange(0, held + 1), spare=held + _spread(rng, 1, 500))
    return c


def _lens(case):
    """(T, L) of the case's sequences: whole numbers of the case alone."""
    r = random.Random(case["lens"])
    L = [r.randint(case["lmin"], case["lmax"]) for _ in range(case["B"])]
    T = [min(l, r.randint(case.get("tmin", 0), case.get("tmax", 0))) for l in L]
    return T, L


def _pages_of(case):
    return sum(-(-l // case["page"]) for l in _lens(case)[1])


def _visible(t, l, w):
    """(query, key) pairs of t new tokens over l cached ones, and the keys that any of them sees."""
    if w <= 0 or w >= l:
        return t * (l - t) + t * (t + 1) // 2, l
    pairs = sum(min(w, l - t + i + 1) for i in range(t))
    return pairs, min(l, w + t - 1)


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["B"] * (case["Hq"] + case["Hkv"]) * case["N"]
        return {"bytes": 4 * n * case["d"] + 4 * case["N"], "flops": 3 * n * case["rot"]}
    T, L = _lens(case)
    if op == "attend":
        seen = [_visible(t, l, case["window"]) for t, l in zip(T, L)]
        rows = sum(T) * case["Hq"]
        return {"bytes": rows * (4 * case["d"] + 4) + 4 * case["Hkv"] * case["d"] * sum(k for _, k in seen),
                "flops": 4 * case["d"] * case["Hq"] * sum(p for p, _ in seen)}
    if op == "append":
        n = sum(T) * (case["Hq"] + 2 * case["Hkv"]) * case["d"]
        return {"bytes": 4 * n, "flops": 3 * sum(T) * (case["Hq"] + case["Hkv"]) * case["rot"]}
    page_bytes = 2 * case["layers"] * case["Hkv"] * case["page"] * case["d"] * 2
    width = -(-2 * case["lmax"] // case["page"]) + 1
    if op == "update":
        P, source, add = _step(case)
        first = {}
        for b, s in enumerate(source):
            if s >= 0 and (s not in first or s == b):
                first[s] = b
        copies = sum(s >= 0 and first[s] != b and L[s] % case["page"] > 0 for b, s in enumerate(source))
        return {"bytes": 8 * P + 8 * case["B"] * width + 2 * copies * page_bytes, "flops": 0}
    P = _pages_of(case) + case["spare"]
    return {"bytes": 8 * P + 8 * case["B"] * width + 2 * case["moves"] * page_bytes, "flops": 0}


def _step(case):
    """(pages of the pool, source row of each next row, tokens that each grows by)."""
    T, L = _lens(case)
    r = random.Random(case["lens"] + 1)
    B = case["B"]
    if case["take"] == "beams":  # groups of up to 8 beams, each going on from a beam of its group
        source = [min(B - 1, b - b % 8 + r.randrange(8)) for b in range(B)]
        add = [1] * B
    else:  # most rows go on; some end and make room for new prompts; some fork
        source, add = [], []
        for b in range(B):
            x = r.random()
            source.append(b if x < 0.8 else -1 if x < 0.95 else r.randrange(B))
            add.append(1 if source[b] >= 0 else r.randint(1, case["lmax"]))
    most = 2 * B if case["take"] == "beams" else B * -(-2 * case["lmax"] // case["page"])
    return _pages_of(case) + most + 8, source, add


# ------------------------------------------------------------------ the inputs

def _ints(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _cu(T):
    out = [0]
    for t in T:
        out.append(out[-1] + t)
    return out


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _table(L, page, width, ids):
    """Rows of page ids, in the order of `ids` (a GPU tensor), -1 behind a row's last page."""
    n = [-(-l // page) for l in L]
    at, rows = _ints(_cu(n)), _ints(n)
    j = torch.arange(width, device="cuda", dtype=torch.int32)
    slot = (at[:-1, None] + j).clamp(max=max(at.numel() and sum(n) - 1, 0))
    return torch.where(j < rows[:, None], ids[slot.long()].to(torch.int32), -1).contiguous()


def _turns(case):
    """Turns a position adds to each pair's angle (angle / 2 pi), 64 bits, and the amplitude."""
    rot, s = case["rot"], case["scaling"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    amp = 1.0
    if s == "linear":
        f = f / 4.0
    elif s == "base":
        f = (10000.0 * 4.0 ** (rot / (rot - 2))) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    elif s == "parts":  # pairs that turn often stay, those that turn seldom are interpolated
        low = rot * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000.0))
        high = rot * math.log(4096 / (1 * 2 * math.pi)) / (2 * math.log(10000.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / 16.0 * ramp + f * (1 - ramp)
        amp = 0.1 * math.log(16.0) + 1.0
    elif s == "bands":  # long wavelengths are interpolated, with a smooth band between
        wave = 2 * math.pi / f
        mix = ((8192 / wave - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = (1 - mix) * f / 8.0 + mix * f
    return f / (2 * math.pi), amp


def prepare(case, seed):
    g, dt, op = _gen(seed), TYPES[case["dtype"]], case["op"]

    def rand(*shape):
        return torch.randn(shape, device="cuda", dtype=dt, generator=g)

    st = dict(case=case, op=op)
    d, Hkv = case["d"], case["Hkv"]
    if op == "rope":
        turns, amp = _turns(case)
        st.update(q=rand(case["B"], case["Hq"], case["N"], d), k=rand(case["B"], Hkv, case["N"], d),
                  pos=torch.arange(case["first"], case["first"] + case["N"], device="cuda", dtype=torch.int32),
                  turns=turns.cuda(), amp=amp)
        return st
    T, L = _lens(case)
    page, B = case["page"], case["B"]
    width = -(-2 * case["lmax"] // page) + 1
    if op in ("attend", "append"):
        total, held = sum(T), _pages_of(case)
        P = held + held // 8 + 3
        ids = torch.randperm(P, device="cuda", generator=g)
        st.update(kpages=rand(P, Hkv, page, d), vpages=rand(P, Hkv, page, d), table=_table(L, page, width, ids),
                  cu=_ints(_cu(T)), lens=_ints(L), max_q=max(T), lmax=max(L))
        if op == "attend":
            st.update(q=rand(total, case["Hq"], d))
        else:  # q, k and v as one projection gives them: side by side in a token's row
            turns, amp = _turns(case)
            qkv = rand(total, case["Hq"] + 2 * Hkv, d)
            st.update(q=qkv[:, :case["Hq"]], k=qkv[:, case["Hq"]:case["Hq"] + Hkv], v=qkv[:, case["Hq"] + Hkv:],
                      turns=turns.cuda(), amp=amp)
        return st
    shape = (case["layers"], None, Hkv, page, d)
    if op == "update":
        P, source, add = _step(case)
        ids = torch.randperm(P, device="cuda", generator=g)
        table = _table(L, page, width, ids)
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        refs[ids[:_pages_of(case)]] = 1
        st.update(source=_ints(source), add=_ints(add))
    else:
        held, moves = _pages_of(case), case["moves"]
        P = held + case["spare"]
        low = torch.randperm(held, device="cuda", generator=g)[:held - moves]
        high = held + torch.randperm(P - held, device="cuda", generator=g)[:moves]
        ids = torch.cat([low, high])[torch.randperm(held, device="cuda", generator=g)]
        table = _table(L, page, width, ids)
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        refs[ids] = 1
    st.update(kpages=rand(shape[0], P, *shape[2:]), vpages=rand(shape[0], P, *shape[2:]), table=table,
              lens=_ints(L), refs=refs)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case, op = st["case"], st["op"]
    if own:
        eta = _lib()
        if op == "attend":
            return eta.attn_paged(st["q"], st["kpages"], st["vpages"], st["table"], st["cu"], st["lens"],
                                  max_q=st["max_q"], window=case["window"])
        if op == "rope":
            fn = eta.attn_rope_bwd if case["grad"] else eta.attn_rope
            return fn(st["q"], st["k"], st["pos"], st["turns"], amp=st["amp"], interleaved=case["interleaved"])
        if op == "append":
            q = eta.attn_rope_append(st["q"], st["k"], st["v"], st["kpages"], st["vpages"], st["table"], st["cu"],
                                     st["lens"], st["turns"], amp=st["amp"], interleaved=case["interleaved"])
            return q, st["kpages"], st["vpages"]
        if op == "update":
            table, lens, refs, info = eta.attn_pages_update(st["kpages"], st["vpages"], st["table"], st["lens"],
                                                            st["refs"], st["source"], st["add"])
            return table, lens, refs, info, st["kpages"], st["vpages"]
        table, refs, info = eta.attn_pages_compact(st["kpages"], st["vpages"], st["table"], st["lens"], st["refs"])
        return table, refs, info, st["kpages"], st["vpages"]
    return {"attend": _attend, "rope": _rope, "append": _append, "update": _update, "compact": _compact}[op](st)


def _attend(st):
    q, kp, vp, table, cu, lens = (st[n] for n in ("q", "kpages", "vpages", "table", "cu", "lens"))
    case = st["case"]
    total, Hq, d = q.shape
    P, Hkv, page, _ = kp.shape
    B, Tm, Lm = lens.numel(), st["max_q"], st["lmax"]
    T, L = (cu[1:] - cu[:-1]).long(), lens.long()
    j = torch.arange(Lm, device="cuda")
    i = torch.arange(Tm, device="cuda")
    at = table.long()[:, j // page].clamp(min=0)                     # [B, Lm]
    k = kp[at, :, j % page].float()                                  # [B, Lm, Hkv, d]
    v = vp[at, :, j % page].float()
    rows = (cu[:-1].long()[:, None] + i).clamp(max=total - 1)
    qs = q[rows].float().view(B, Tm, Hkv, Hq // Hkv, d)
    s = torch.matmul(qs.permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d), k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    last = (L - T)[:, None] + i                                      # [B, Tm]: the position of each new token
    see = (j <= last[..., None]) & (j < L[:, None, None])
    if case["window"] > 0:
        see = see & (j > last[..., None] - case["window"])
    s = s.view(B, Hkv, Hq // Hkv, Tm, Lm).masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, Lm), v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, Tm, d) / l
    lse = (m + l.log()).squeeze(-1)                                  # [B, Hkv, G, Tm]
    n = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].long(), n, right=True)
    t = n - cu.long()[b]
    return o[b, :, :, t].reshape(total, Hq, d).to(q.dtype), lse[b, :, :, t].reshape(total, Hq)


def _turn(x, angle, amp, rot, interleaved):
    """x [..., d] with its first `rot` values turned by angle [..., rot / 2]."""
    c, s = (angle.cos() * amp).float(), (angle.sin() * amp).float()
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _rope(st):
    case = st["case"]
    angle = st["pos"].double()[:, None] * st["turns"] * (2 * math.pi)
    if case["grad"]:
        angle = -angle
    return tuple(_turn(st[n], angle, st["amp"], case["rot"], case["interleaved"]) for n in ("q", "k"))


def _append(st):
    case, cu, kp, vp = st["case"], st["cu"].long(), st["kpages"], st["vpages"]
    page = kp.shape[2]
    n = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], n, right=True)
    pos = st["lens"].long()[b] - cu[b + 1] + n
    angle = (pos.double()[:, None] * st["turns"] * (2 * math.pi))[:, None]
    q = _turn(st["q"], angle, st["amp"], case["rot"], case["interleaved"])
    k = _turn(st["k"], angle, st["amp"], case["rot"], case["interleaved"])
    at = st["table"].long()[b, pos // page]
    kp[at, :, pos % page] = k
    vp[at, :, pos % page] = st["v"]
    return q, kp, vp


def _update(st):
    table, lens, refs, kp = st["table"].long(), st["lens"].long(), st["refs"].long(), st["kpages"]
    source, add = st["source"].long(), st["add"].long()
    page, P, width, B = kp.shape[3], refs.numel(), table.shape[1], lens.numel()
    row = torch.arange(B, device="cuda")
    j = torch.arange(width, device="cuda")
    live = source >= 0
    s = source.clamp(min=0)
    L = torch.where(live, lens[s], 0)
    # The row that goes on in its source's own last page: the source itself, or the first that takes it over.
    first = torch.full((B + 1,), B, device="cuda").scatter_reduce(0, torch.where(live, s, B), row, "amin")[:B]
    first = torch.where(source == row, row, first)
    keeps = live & (first[s] == row)
    full, held = L // page, -(-L // page)
    kept = torch.where(keeps, held, full)
    longer = L + add
    want = -(-longer // page)
    old = (j < (-(-lens // page))[:, None])
    refs = refs.scatter_add(0, table.clamp(min=0).flatten(), -old.flatten().long())
    stay = j < kept[:, None]
    refs = refs.scatter_add(0, table[s].clamp(min=0).flatten(), stay.flatten().long())
    # The lowest free pages, in order, to the rows' new slots, in order.
    empty = refs <= 0
    order = torch.where(empty, empty.cumsum(0) - 1, P)
    lowest = torch.full((P + 1,), -1, device="cuda").scatter_(0, order, torch.arange(P, device="cuda"))
    need = want - kept
    rank = (need.cumsum(0) - need)[:, None] + (j - kept[:, None])
    fresh = ~stay & (j < want[:, None])
    new = torch.where(fresh, lowest[rank.clamp(0, P)], torch.where(stay, table[s], -1))
    refs = refs.scatter_add(0, new.clamp(min=0).flatten(), fresh.flatten().long())
    info = torch.stack([(need.sum() - empty.sum()).clamp(min=0), (longer > width * page).sum()])
    copy = live & ~keeps & (held > full)
    at = full.clamp(max=width - 1)
    to, of = new[row, at][copy], table[s, at][copy]
    kp[:, to] = kp[:, of]
    st["vpages"][:, to] = st["vpages"][:, of]
    i32 = torch.int32
    return new.to(i32), longer.to(i32), refs.to(i32), info.to(i32), kp, st["vpages"]


def _compact(st):
    table, refs, kp = st["table"].long(), st["refs"].long(), st["kpages"]
    page, P, width = kp.shape[3], refs.numel(), table.shape[1]
    n = (refs > 0).sum()
    at = torch.arange(P, device="cuda")
    of = ((refs > 0) & (at >= n)).nonzero().squeeze(1)   # live pages behind the first n, in order
    to = ((refs <= 0) & (at < n)).nonzero().squeeze(1)   # free pages among the first n, in order
    moved = at.scatter(0, of, to)
    kp[:, to] = kp[:, of]
    st["vpages"][:, to] = st["vpages"][:, of]
    held = torch.arange(width, device="cuda") < (-(-st["lens"].long() // page))[:, None]
    new = torch.where(held, moved[table.clamp(min=0)], -1)
    count = torch.where(at < n, refs, 0).scatter(0, to, refs[of])
    info = torch.stack([n, torch.full_like(n, of.numel())])
    return new.to(torch.int32), count.to(torch.int32), info.to(torch.int32), kp, st["vpages"]


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        return _exact_attend(st)
    if op == "rope":
        sign = -1.0 if case["grad"] else 1.0
        pos = st["pos"].double()
        return tuple(_exact_turn(st[n].double(), pos, st, sign) for n in ("q", "k"))
    if op == "append":
        kp, vp = st["kpages"].double(), st["vpages"].double()
        q = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        T, L = _lens(case)
        at = 0
        page = case["page"]
        for b, (t, l) in enumerate(zip(T, L)):
            if t == 0:
                continue
            pos = torch.arange(l - t, l, device="cuda")
            part = slice(at, at + t)
            where = st["table"][b].long()[pos // page]
            q[part] = _exact_turn(st["q"][part].double().transpose(0, 1), pos.double(), st, 1.0).transpose(0, 1)
            kp[where, :, pos % page] = _exact_turn(st["k"][part].double().transpose(0, 1), pos.double(), st,
                                                   1.0).transpose(0, 1)
            vp[where, :, pos % page] = st["v"][part].double()
            at += t
        return q, kp, vp
    if op == "update":
        return _exact_update(st)
    return _exact_compact(st)


def _exact_attend(st):
    case, q, kp, vp = st["case"], st["q"], st["kpages"], st["vpages"]
    total, Hq, d = q.shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    o = torch.zeros((total, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((total, Hq), -math.inf, dtype=torch.float64, device="cuda")
    T, L = _lens(case)
    at = 0
    for b, (t, l) in enumerate(zip(T, L)):
        pages = st["table"][b, :-(-l // page)].long()
        w = case["window"] if case["window"] > 0 else l
        j, pos = torch.arange(l, device="cuda"), torch.arange(l - t, l, device="cuda")
        see = (j[None] <= pos[:, None]) & (j[None] > pos[:, None] - w)
        for g in range(Hkv):
            k = kp[pages, g].reshape(-1, d)[:l].double()
            v = vp[pages, g].reshape(-1, d)[:l].double()
            for h in range(g * G, g * G + G):
                s = (q[at:at + t, h].double() @ k.T) / math.sqrt(d)
                s = torch.where(see, s, -math.inf)
                e = torch.logsumexp(s, -1)
                o[at:at + t, h] = torch.exp(s - e[:, None]) @ v
                lse[at:at + t, h] = e
        at += t
    return o, lse


def _exact_turn(x, pos, st, sign):
    """x [..., N, d] in 64 bits: pair p of position n times amp e^(i sign angle)."""
    rot = st["case"]["rot"]
    f = _turns(st["case"])[0].cuda()
    a = 2 * math.pi * torch.remainder(pos[:, None] * f, 1.0)
    z = torch.polar(torch.full_like(a, st["amp"]), sign * a)
    y = x.clone()
    if st["case"]["interleaved"]:
        r = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = r.real, r.imag
    else:
        r = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = r.real, r.imag
    return y


def _exact_update(st):
    """Row by row on the host: whole numbers, and pages that only move."""
    table, lens, refs = st["table"].tolist(), st["lens"].tolist(), st["refs"].tolist()
    source, add = st["source"].tolist(), st["add"].tolist()
    page, width = st["case"]["page"], len(table[0])
    for b, l in enumerate(lens):
        for p in table[b][:-(-l // page)]:
            refs[p] -= 1
    keeper = {}
    for b, s in enumerate(source):
        if s >= 0 and (s not in keeper or s == b):
            keeper[s] = b
    rows, kept = [], []
    for b, s in enumerate(source):
        l = lens[s] if s >= 0 else 0
        n = -(-l // page) if s >= 0 and keeper[s] == b else l // page
        rows.append(table[s][:n] if s >= 0 else [])
        kept.append(n)
        for p in rows[-1]:
            refs[p] += 1
    free = [p for p, r in enumerate(refs) if r <= 0]
    at, kp, vp, longer = 0, st["kpages"].double(), st["vpages"].double(), []
    for b, s in enumerate(source):
        l = lens[s] if s >= 0 else 0
        longer.append(l + add[b])
        want = -(-longer[-1] // page)
        new = free[at:at + want - kept[b]]
        at += len(new)
        if kept[b] < -(-l // page):
            kp[:, new[0]] = kp[:, table[s][kept[b]]]
            vp[:, new[0]] = vp[:, table[s][kept[b]]]
        for p in new:
            refs[p] += 1
        rows[b] = rows[b] + new + [-1] * (width - want)
    return _ints(rows), _ints(longer), _ints(refs), _ints([0, 0]), kp, vp


def _exact_compact(st):
    table, lens, refs = st["table"].tolist(), st["lens"].tolist(), st["refs"].tolist()
    page = st["case"]["page"]
    n = sum(r > 0 for r in refs)
    of = [p for p in range(n, len(refs)) if refs[p] > 0]
    to = [p for p in range(n) if refs[p] <= 0]
    kp, vp = st["kpages"].double(), st["vpages"].double()
    for a, b in zip(of, to):
        kp[:, b], vp[:, b] = kp[:, a], vp[:, a]
        refs[b] = refs[a]
    moved = dict(zip(of, to))
    rows = [[moved.get(p, p) if j < -(-l // page) else -1 for j, p in enumerate(r)] for r, l in zip(table, lens)]
    return _ints(rows), _ints(refs[:n] + [0] * (len(refs) - n)), _ints([n, len(of)]), kp, vp
