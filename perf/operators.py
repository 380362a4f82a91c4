"""Cases of the paged serving operators: the page plan (block tables and slot maps built on
the GPU), the q/k norm + rotary + cache append, and one-token attention over the paged cache.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a
case's inputs, ``run()`` is one pass (the plain torch form, or the framework's call where
``own`` is true), ``work()`` its bytes and FLOPs, ``exact()`` the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a small server: every running request gets one token, one in
        # eight takes a new page, a few have finished and give theirs back
        dict(name="plan decode 64", op="plan", n=64, page=16, lo=1, hi=4096, tokens=64,
             finished=0.05, fresh=0.0, spread=1),
        # a mixed step: decode rows, finished requests and chunks of prompts side by side,
        # more asked for than the step's token budget holds
        dict(name="plan mixed 509", op="plan", n=509, page=32, lo=1, hi=16384, tokens=8192,
             finished=0.1, fresh=0.08, spread=2),
        # a batch start: thousands of prompts placed at once
        dict(name="plan prompts 4096", op="plan", n=4096, page=16, lo=0, hi=128, tokens=262144,
             finished=0.02, fresh=0.9, spread=3),
        # the model's attention layer, one new token of 64 sequences (three-axis positions)
        dict(name="append decode 64", op="append", t=64, hq=24, hkv=4, d=256, rope=64,
             inter=False, axes=3, x="bf16", cache="fp16", page=64, heads_first=False,
             norm=True, scaled=False, far=200000, pad=0),
        # the same layer on a prompt chunk of the benchmark's length
        dict(name="append prompt 8192", op="append", t=8192, hq=24, hkv=4, d=256, rope=64,
             inter=False, axes=3, x="bf16", cache="fp16", page=64, heads_first=False,
             norm=True, scaled=False, far=0, pad=0),
        # another layout: head dim 128 turned whole, adjacent pairs, a scaled long context,
        # an odd count of tokens with padding rows behind them, heads before tokens in a page
        dict(name="append interleaved 1999", op="append", t=1999, hq=32, hkv=8, d=128, rope=128,
             inter=True, axes=1, x="bf16", cache="bf16", page=16, heads_first=True,
             norm=True, scaled=True, far=100000, pad=31),
        # plain rotary of fp32 activations on part of a narrow head, no norm
        dict(name="append fp32 part 333", op="append", t=333, hq=8, hkv=2, d=64, rope=20,
             inter=False, axes=1, x="fp32", cache="fp16", page=24, heads_first=False,
             norm=False, scaled=False, far=30000, pad=0),
        # latency: a few short conversations
        dict(name="decode 8 short", op="decode", n=8, lo=1, hi=300, hq=24, hkv=4, d=256,
             page=16, cache="fp16", heads_first=False, gate=True, lse=False, out="bf16",
             spread=4),
        # one request with a long context: all the work lies along one cache
        dict(name="decode 1 x 131072", op="decode", n=1, lo=131071, hi=131071, hq=24, hkv=4,
             d=256, page=64, cache="fp16", heads_first=False, gate=True, lse=False, out="bf16",
             spread=5),
        # the benchmark's decode batch
        dict(name="decode 256 x 4096", op="decode", n=256, lo=4097, hi=4097, hq=24, hkv=4,
             d=256, page=64, cache="fp16", heads_first=False, gate=True, lse=False, out="bf16",
             spread=6),
        # ragged traffic: lengths over four decades, head dim 128, pages that end inside a
        # tile, sums returned for a later join
        dict(name="decode ragged 128", op="decode", n=128, lo=1, hi=16384, hq=32, hkv=8, d=128,
             page=16, cache="bf16", heads_first=True, gate=False, lse=True, out="bf16",
             spread=7),
        # no sharing of key-value heads, narrow heads, a page size that is no power of two
        dict(name="decode heads 16:16", op="decode", n=61, lo=1, hi=3000, hq=16, hkv=16, d=64,
             page=48, cache="fp16", heads_first=False, gate=False, lse=False, out="fp32",
             spread=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode"])
    page = rng.choice([1, 7, 8, 16, 24, 32, 48, 64, 128, 256])
    if op == "plan":
        n = _log_int(rng, 1, 4096)
        return dict(op=op, n=n, page=max(page, 7), lo=rng.choice([0, 1]),
                    hi=_log_int(rng, 16, 16384 if n <= 512 else 512),
                    tokens=_log_int(rng, n, 262144), finished=rng.choice([0.0, 0.05, 0.3]),
                    fresh=rng.choice([0.0, 0.1, 0.9]), spread=rng.randrange(1 << 20))
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "append":
        half = [r for r in (10, 32, d // 4, d // 2) if r <= d // 2]
        return dict(op=op, t=_log_int(rng, 1, 8192 if hkv * g * d <= 6144 else 4096), hq=hkv * g,
                    hkv=hkv, d=d, rope=2 * rng.choice(half), inter=rng.random() < 0.5,
                    axes=rng.choice([1, 3]), x=rng.choice(["bf16", "fp16", "fp32"]),
                    cache=rng.choice(["bf16", "fp16"]), page=page,
                    heads_first=rng.random() < 0.5, norm=rng.random() < 0.7,
                    scaled=rng.random() < 0.5, far=rng.choice([0, 1000, 250000]),
                    pad=rng.choice([0, 0, 5]))
    n = _log_int(rng, 1, 256)
    most = min(131072, (1 << 30) // (n * hkv * d))
    hi = _log_int(rng, 1, max(1, most))
    return dict(op=op, n=n, lo=rng.choice([0, 1, hi]), hi=hi, hq=hkv * g, hkv=hkv, d=d,
                page=page, cache=rng.choice(["bf16", "fp16"]), heads_first=rng.random() < 0.5,
                gate=rng.random() < 0.5, lse=rng.random() < 0.5,
                out=rng.choice(["bf16", "fp16", "fp32"]), spread=rng.randrange(1 << 20))


# ----------------------------------------------------------------------- inputs --

def _lengths(c):
    """Lengths of a case, spread over the logarithm of [lo, hi]; the same for every seed."""
    r = random.Random(c["spread"])
    lo, hi = c["lo"], c["hi"]
    got = [lo if lo == hi or (lo == 0 and r.random() < 0.1) else _log_int(r, max(lo, 1), hi)
           for _ in range(c["n"])]
    got[0] = hi
    return got


def _plan_lengths(c):
    """(lens, want): decode rows grow by one, finished ones go to zero, fresh ones get a
    prompt or a chunk of one."""
    lens = _lengths(c)
    r = random.Random(c["spread"] + 1)
    want = []
    for i, n in enumerate(lens):
        u = r.random()
        if u < c["finished"]:
            want.append(0)
        elif u < c["finished"] + c["fresh"]:
            want.append(n + _log_int(r, 1, max(2, 2 * c["tokens"] // max(1, int(c["n"] * c["fresh"])))))
        else:
            want.append(n + 1)
    return lens, want


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(g, pages, c):
    """A cache view [pages, page, hkv, d]; with heads_first a page holds head after head."""
    dt, p, h, d = DT[c["cache"]], c["page"], c["hkv"], c["d"]
    shape = (pages, h, p, d) if c["heads_first"] else (pages, p, h, d)
    t = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    return t.transpose(1, 2) if c["heads_first"] else t


def prepare(case, seed):
    c = case
    g = _gen(seed)
    if c["op"] == "plan":
        lens, want = _plan_lengths(c)
        order = torch.randperm(c["n"], generator=g, device="cuda")
        lens = torch.tensor(lens, device="cuda")[order]
        want = torch.tensor(want, device="cuda")[order]
        p = c["page"]
        held = (lens + p - 1) // p
        width = int(torch.maximum(held, (want + p - 1) // p).max())
        total = int(held.sum())
        # room for most, not always all, of what the step asks for
        pool = total + int(((want - lens).clamp(min=0) // p + 1).sum() * 9 // 10) + 1
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["n"], width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda")[None] < held[:, None]] = ids[:total]
        free = torch.zeros(pool, dtype=torch.int32, device="cuda")
        free[:pool - total] = ids[total:]
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(c=c, lens=lens.to(torch.int32), want=want.to(torch.int32), table=table,
                    free=free, count=torch.tensor([pool - total], **i32),
                    out=dict(new_lens=torch.empty(c["n"], **i32),
                             cu_new=torch.empty(c["n"] + 1, **i32),
                             slot_map=torch.empty(c["tokens"], **i32),
                             positions=torch.empty(c["tokens"], **i32),
                             new_count=torch.empty(1, **i32), info=torch.empty(4, **i32)))
    if c["op"] == "append":
        t, d, x = c["t"], c["d"], DT[c["x"]]
        pages = (t - c["pad"] + c["page"] - 1) // c["page"] + 3 if t > c["pad"] else 3
        # q, k and v are views of one projection's rows
        rows = _normal(g, (t, (c["hq"] + 2 * c["hkv"]) * d), x)
        q, k, v = (a.unflatten(1, (-1, d)) for a in
                   rows.split([c["hq"] * d, c["hkv"] * d, c["hkv"] * d], dim=1))
        slots = torch.randperm(pages * c["page"], generator=g, device="cuda")
        slots = slots[:t].to(torch.int32) if slots.numel() >= t else torch.cat(
            [slots, slots.new_full((t - slots.numel(),), -1)]).to(torch.int32)
        if c["pad"]:
            slots[max(0, t - c["pad"]):] = -1
        pos = torch.arange(t, device="cuda") + int(torch.randint(
            c["far"] + 1, (1,), generator=g, device="cuda"))
        if c["axes"] == 3:
            pos = torch.stack([pos, pos // 2, pos % 97])
        i = torch.arange(c["rope"] // 2, dtype=torch.float64, device="cuda")
        f = 1e7 ** (-2 * i / c["rope"])
        if c["scaled"]:                       # interpolation by parts over an 8 times longer context
            turns = (8192 * f / (2 * math.pi) - 1) / 31
            keep = turns.clamp(0, 1)
            f = f * (keep + (1 - keep) / 8)
        w = [(1 + 0.1 * _normal(g, (d,), torch.float32)).to(torch.bfloat16) if c["norm"] else None
             for _ in range(2)]
        return dict(c=c, q=q, k=k, v=v, slots=slots, pos=pos.to(torch.int32).contiguous(), f=f,
                    wq=w[0], wk=w[1], mscale=0.1 * math.log(8) + 1 if c["scaled"] else 1.0,
                    kc=_cache(g, pages, c), vc=_cache(g, pages, c),
                    qo=torch.empty((t, c["hq"], d), dtype=DT[c["cache"]],
                                   device="cuda").normal_(generator=g))
    lens = torch.tensor(_lengths(c), device="cuda")
    lens = lens[torch.randperm(c["n"], generator=g, device="cuda")]
    p, n = c["page"], c["n"]
    held = (lens + p - 1) // p
    width = max(1, (c["hi"] + p - 1) // p)
    pages = int(held.sum()) + 2
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda")[None] < held[:, None]
    table[used] = ids[:pages - 2]
    kc, vc = _cache(g, pages, c), _cache(g, pages, c)
    # what lies behind a sequence in its last page was never written
    off = torch.arange(p, device="cuda")[None]
    last = table.long().gather(1, (held - 1).clamp(min=0)[:, None])
    dead = (off >= (lens - (held - 1) * p)[:, None]) & (held > 0)[:, None]
    at = (last.expand(-1, p)[dead], off.expand(n, p)[dead])
    kc[at] = float("nan")
    vc[at] = float("inf")
    dt = DT[c["cache"]]
    return dict(c=c, q=_normal(g, (n, c["hq"], c["d"]), dt), kc=kc, vc=vc, table=table,
                lens=lens.to(torch.int32),
                gate=_normal(g, (n, c["hq"], c["d"]), torch.bfloat16) if c["gate"] else None)


# ------------------------------------------------------------------ plain forms --

def _ceil(a, p):
    return (a + p - 1) // p


def _plan_plain(s):
    c, table, free = s["c"], s["table"], s["free"]
    p, cap = c["page"], table.shape[1] * c["page"]
    pool = free.numel()
    lens, want, dev = s["lens"].long(), s["want"].long(), table.device
    count = s["count"].long().clamp(0, pool)
    fine = (lens >= 0) & (lens <= cap) & (want >= 0) & (want <= cap)
    held, goal = _ceil(lens, p), _ceil(want, p)
    col = torch.arange(table.shape[1], device=dev)[None]
    # pages given back, in request order, on top of the stack
    back = (fine & (want < lens))[:, None] & (col >= goal[:, None]) & (col < held[:, None])
    given = table[back]
    room = pool - int(count)
    given = given[:room]
    stack = torch.cat([free[:int(count)], given])
    # growth in request order, as long as pages and tokens last
    grow = fine & (want > lens)
    need = torch.where(grow, goal - held, 0)
    more = torch.where(grow, want - lens, 0)
    grant = grow & (need.cumsum(0) <= stack.numel()) & (more.cumsum(0) <= c["tokens"])
    need, more = need * grant, more * grant
    new = grant[:, None] & (col >= held[:, None]) & (col < goal[:, None])
    taken = int(need.sum())
    table[new] = stack.flip(0)[:taken]
    left = stack.numel() - taken
    if left > int(count):
        free[int(count):left] = stack[int(count):left]
    new_lens = torch.where(grant | (fine & (want < lens)), want, lens)
    cu = torch.cat([more.new_zeros(1), more.cumsum(0)])
    t = torch.arange(c["tokens"], device=dev)
    n = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["n"] - 1)
    live = t < cu[-1]
    pos = torch.where(live, lens[n] + t - cu[n], 0)
    slot = torch.where(live, table[n, pos // p].long() * p + pos % p, -1)
    asked = want != lens
    refused = (asked & ~grant & ~(fine & (want < lens))).sum()
    info = torch.stack([cu[-1], need.sum(), torch.tensor(given.numel(), device=dev), refused])
    i32 = torch.int32
    return dict(new_lens=new_lens.to(i32), cu_new=cu.to(i32), slot_map=slot.to(i32),
                positions=pos.to(i32), new_count=torch.tensor([left], dtype=i32, device=dev),
                info=info.to(i32), table=table, free=free)


def _norm_rope_plain(x, w, cos, sin, rope, inter, eps=1e-6):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    r, rest = x[..., :rope], x[..., rope:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else r.chunk(2, dim=-1)
    turned = (a * cos - b * sin, b * cos + a * sin)
    r = torch.stack(turned, dim=-1).flatten(-2) if inter else torch.cat(turned, dim=-1)
    return torch.cat([r, rest], dim=-1)


def _append_plain(s):
    c = s["c"]
    pairs = torch.arange(c["rope"] // 2, device="cuda")
    pos = s["pos"][pairs % 3].T if c["axes"] == 3 else s["pos"][:, None]
    angle = pos.double() * s["f"]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    live = (s["slots"] >= 0) & (s["slots"] < s["kc"].shape[0] * c["page"])
    slot = s["slots"][live].long()
    at = (slot // c["page"], slot % c["page"])
    q = _norm_rope_plain(s["q"], s["wq"], cos, sin, c["rope"], c["inter"])
    k = _norm_rope_plain(s["k"], s["wk"], cos, sin, c["rope"], c["inter"])
    s["qo"][live] = q[live].to(s["qo"].dtype)
    s["kc"][at] = k[live].to(s["kc"].dtype)
    s["vc"][at] = s["v"][live].to(s["vc"].dtype)
    return dict(q=s["qo"], k_cache=s["kc"], v_cache=s["vc"])


def _decode_plain(s):
    c = s["c"]
    n, h, d, p = c["n"], c["hkv"], c["d"], c["page"]
    at = s["table"].long().clamp(0, s["kc"].shape[0] - 1)
    k = s["kc"][at].flatten(1, 2).float()                      # [n, tokens, h, d]
    live = torch.arange(k.shape[1], device="cuda")[None] < s["lens"][:, None]
    q = s["q"].float().unflatten(1, (h, -1))
    x = torch.einsum("nhgd,nthd->nhgt", q, k) * d ** -0.5
    del k
    x = x.masked_fill(~live[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == float("-inf"), 0)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = s["vc"][at].flatten(1, 2).float().masked_fill(~live[..., None, None], 0)
    o = torch.einsum("nhgt,nthd->nhgd", x, v) / total
    o = o.masked_fill(total == 0, 0).flatten(1, 2)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    out = dict(o=o.to(DT[c["out"]]))
    if c["lse"]:
        out["lse"] = (top + torch.log(total)).flatten(1)
    return out


# ---------------------------------------------------------------------- one pass --

def run(state):
    s, c = state, state["c"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "decode": _decode_plain}[c["op"]](s)
    import gated_delta_rule_106_b200 as gdn
    if c["op"] == "plan":
        gdn.gdn_page_plan(s["lens"], s["want"], s["table"], s["free"], s["count"], c["page"],
                          **s["out"])
        return dict(s["out"], table=s["table"], free=s["free"])
    if c["op"] == "append":
        gdn.gdn_qk_norm_rope(s["q"], s["k"], s["v"], s["kc"], s["vc"], slot_map=s["slots"],
                             q_norm_w=s["wq"], k_norm_w=s["wk"], positions=s["pos"],
                             inv_freq=s["f"], interleaved=c["inter"], rope_scale=s["mscale"],
                             q_out=s["qo"])
        return dict(q=s["qo"], k_cache=s["kc"], v_cache=s["vc"])
    lse = torch.empty((c["n"], c["hq"]), dtype=torch.float32, device="cuda") if c["lse"] else None
    o = gdn.gdn_paged_attention_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                       gate=s["gate"], o_dtype=DT[c["out"]], lse=lse)
    return dict(o=o, lse=lse) if c["lse"] else dict(o=o)


# -------------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "plan":
        lens, want = _plan_lengths(c)
        p = c["page"]
        moved = sum(abs(_ceil(w, p) - _ceil(n, p)) for n, w in zip(lens, want))
        # lengths in and out, prefix sums, slots and positions of the budget, pages moved
        return dict(bytes=4 * (4 * c["n"] + 2 * c["tokens"] + 2 * moved), flops=0)
    if c["op"] == "append":
        size = 4 if c["x"] == "fp32" else 2
        live = max(1, c["t"] - c["pad"])
        values = live * (c["hq"] + 2 * c["hkv"]) * c["d"]
        turned = live * (c["hq"] + c["hkv"])
        return dict(bytes=values * (size + 2) + 4 * c["t"] * (1 + c["axes"]),
                    flops=turned * (4 * c["d"] * c["norm"] + 3 * c["rope"]))
    tokens = sum(_lengths(c))
    heads = c["n"] * c["hq"] * c["d"]
    size = 4 if c["out"] == "fp32" else 2
    return dict(bytes=4 * tokens * c["hkv"] * c["d"] + heads * (2 + size + 2 * c["gate"])
                + 4 * tokens // c["page"] + 4 * c["n"] * (1 + c["lse"] * c["hq"]),
                flops=4 * tokens * c["hq"] * c["d"])


# ------------------------------------------------------------------- in 64 bits --

def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None                                   # whole numbers
    s = prepare(case, seed)
    d = c["d"]
    if c["op"] == "append":
        out = dict(q=s["qo"].double(), k_cache=s["kc"].double(), v_cache=s["vc"].double())
        live = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        slot = s["slots"].double()[live].long()
        page = torch.div(slot, c["page"], rounding_mode="floor")
        half = c["rope"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
        pos = s["pos"].double().reshape(-1, c["t"])
        pos = pos[i % pos.shape[0]].T[live]
        turn = torch.polar(torch.full_like(pos, s["mscale"]), pos * s["f"])[:, None]
        for name, x, w in (("q", s["q"], s["wq"]), ("k_cache", s["k"], s["wk"])):
            x = x[live].to(torch.float64)
            if w is not None:
                x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
            z = torch.complex(x[..., first], x[..., second]) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            if name == "q":
                out["q"][live] = y
            else:
                out[name][page, slot - page * c["page"]] = y
        out["v_cache"][page, slot - page * c["page"]] = s["v"][live].double()
        return out
    o = torch.zeros((c["n"], c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["n"], c["hq"]), float("-inf"), dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for n, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        pages = s["table"][n, : -(-length // c["page"])].tolist()
        pages = torch.tensor(pages, device="cuda")
        k = s["kc"].index_select(0, pages).reshape(-1, c["hkv"], d)[:length].double()
        v = s["vc"].index_select(0, pages).reshape(-1, c["hkv"], d)[:length].double()
        q = s["q"][n].double().reshape(c["hkv"], group, d)
        x = torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(d)
        lse[n] = torch.logsumexp(x, -1).reshape(-1)
        o[n] = torch.bmm(torch.softmax(x, -1), v.transpose(0, 1)).reshape(-1, d)
    if s["gate"] is not None:
        o = o / (1 + torch.exp(-s["gate"].double()))
    return dict(o=o, lse=lse) if c["lse"] else dict(o=o)
