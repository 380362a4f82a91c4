"""GPU: the paged-cache operators (gdn_page_plan, gdn_rope_inv_freq,
gdn_qk_norm_rope, gdn_paged_attention_decode) against plain 64-bit forms
(``tests/_paged.py``), and a server's steps with all of them against the
attention layer's oracle."""
import math

import numpy as np
import pytest
import torch

import gdn_inputs as gi
import oracle
import gated_delta_rule_106_b200 as gdn
import _paged as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
f64 = ref.f64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------- plan --

def plan_state(rng, lens, width, page, spare):
    """A table whose held pages are distinct, and the stack of the others."""
    held = [-(-n // page) for n in lens]
    total = sum(held)
    P = max(1, total + spare)
    ids = rng.permutation(P).tolist()
    table = np.full((len(lens), width), -7, dtype=np.int32)
    at = 0
    for n, h in enumerate(held):
        table[n, :h] = ids[at:at + h]
        at += h
    free = np.full(P, -9, dtype=np.int32)
    free[:P - total] = ids[total:]
    return table, free, P - total


def check_plan(lens, want, table, free, count, page, capacity, **kw):
    t, f = i32(table), i32(free)
    a, b, c = i32(lens).reshape(-1), i32(want).reshape(-1), i32([count])
    t = t.reshape(len(lens), -1)
    r = ref.plan(lens, want, table.tolist(), free.tolist(), count, page, capacity)
    for again in range(2):                       # the same call again: the same result
        got = gdn.gdn_page_plan(a, b, t, f, c, page, token_capacity=capacity, **kw)
        for name in ("new_lens", "cu_new", "slot_map", "positions", "new_count", "info"):
            assert getattr(got, name).tolist() == r[name], (again, name)
        assert t.tolist() == r["table"] and f.tolist() == r["free"], again
    assert a.tolist() == list(lens) and b.tolist() == list(want) and c.tolist() == [count]
    return got, r


@pytest.mark.parametrize("N,page,hi,capacity,spare", [
    (1, 16, 40, 64, 8), (1, 1, 3, 1, 0), (7, 5, 60, 100, 10), (64, 16, 900, 64, 9),
    (33, 32, 400, 3001, 40), (1025, 16, 50, 5000, 300), (2500, 3, 20, 40000, 9000)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan_random_steps(N, page, hi, capacity, spare, seed):
    rng = np.random.default_rng([N, page, seed])
    lens = rng.integers(0, hi + 1, N).tolist()
    kind = rng.integers(0, 5, N)
    want = [n + 1 if k < 2 else 0 if k == 2 else int(rng.integers(0, n + 1)) if k == 3
            else n + int(rng.integers(0, 2 * capacity // N + 2)) for n, k in zip(lens, kind)]
    width = max(1, max(-(-n // page) for n in lens + want))
    table, free, count = plan_state(rng, lens, width, page, spare)
    check_plan(lens, want, table, free, count, page, capacity)


def test_plan_edges():
    rng = np.random.default_rng(3)
    # nothing fits from the second growing request on; a later one without new pages is refused too
    lens, want = [15, 16, 3, 0, 20], [16, 40, 4, 0, 0]
    table, free, count = plan_state(rng, lens, 4, 16, 0)
    _, r = check_plan(lens, want, table, free, count, 16, 8)
    assert r["new_lens"] == [16, 16, 3, 0, 0] and r["info"] == [1, 0, 2, 2]
    # the token budget ends the growth although pages are left
    table, free, count = plan_state(rng, [0, 0, 0], 4, 16, 20)
    _, r = check_plan([0, 0, 0], [5, 4, 1], table, free, count, 16, 8)
    assert r["new_lens"] == [5, 0, 0]
    # returned pages are taken in the same step
    table, free, count = plan_state(rng, [64, 0], 4, 16, 0)
    _, r = check_plan([64, 0], [0, 50], table, free, count, 16, 50)
    assert r["info"] == [50, 4, 4, 0]
    # lengths out of range are refused alone; a full row is not
    table, free, count = plan_state(rng, [0, 0, 0, 10], 2, 8, 9)
    _, r = check_plan([-1, 0, 17, 10], [3, 17, 4, 16], table, free, count, 8, 40)
    assert r["new_lens"] == [-1, 0, 17, 16] and r["info"][3] == 3
    # entries that are no pages give no slot
    free[:count] = [0] * (count - 3) + [-5, 99, 2 ** 31 - 1]
    check_plan([0, 0, 0, 0], [8, 8, 8, 8], table, free, count, 8, 40)
    # a count outside the stack
    for c in (-3, 1000):
        check_plan([0], [5], np.zeros((1, 2), np.int32), np.arange(2, dtype=np.int32), c, 4, 8)
    # returns past the stack's room are dropped
    check_plan([8], [0], np.array([[1, 0]], np.int32), np.arange(2, dtype=np.int32), 1, 4, 8)
    # no requests; no room for tokens
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    got = gdn.gdn_page_plan(e, e, e.reshape(0, 3), i32([4, 5]), i32([2]), 16, token_capacity=5)
    assert got.slot_map.tolist() == [-1] * 5 and got.cu_new.tolist() == [0]
    assert got.new_count.tolist() == [2] and got.info.tolist() == [0, 0, 0, 0]
    table, free, count = plan_state(rng, [3, 9], 2, 8, 1)
    check_plan([3, 9], [4, 0], table, free, count, 8, 0)


def test_plan_strided_table_most_requests_and_graph():
    """A table that is a view of wider rows; the most requests a call takes; a
    captured step replayed on new lengths."""
    rng = np.random.default_rng(5)
    N, page = 16384, 16
    lens = rng.integers(0, 33, N).tolist()
    want = [n + 1 for n in lens]
    table, free, count = plan_state(rng, lens, 3, page, 3000)
    r = ref.plan(lens, want, table.tolist(), free.tolist(), count, page, N + 3)
    wide = torch.full((N, 11), 77, dtype=torch.int32, device=DEV)
    wide[:, 4:7] = i32(table)
    a, w, f, c = i32(lens), i32(want), i32(free), i32([count])
    out = gdn.gdn_page_plan(a, w, wide[:, 4:7], f, c, page, token_capacity=N + 3)
    assert wide[:, 4:7].tolist() == r["table"]
    assert bool((wide[:, :4] == 77).all()) and bool((wide[:, 7:] == 77).all())
    assert out.slot_map.tolist() == r["slot_map"] and f.tolist() == r["free"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        gdn.gdn_page_plan(a, w, wide[:, 4:7], f, c, page, **out._asdict())
        a.copy_(out.new_lens)
        c.copy_(out.new_count)
        w.copy_(out.new_lens + 1)
    torch.cuda.synchronize()
    lens2, table2, free2, count2 = lens, table.tolist(), free.tolist(), count
    for _ in range(3):
        r = ref.plan(lens2, [n + 1 for n in lens2], table2, free2, count2, page, N + 3)
        g.replay()
        assert out.slot_map.tolist() == r["slot_map"] and out.info.tolist() == r["info"]
        lens2, table2, free2, count2 = r["new_lens"], r["table"], r["free"], r["new_count"][0]
    assert wide[:, 4:7].tolist() == table2


# -------------------------------------------------------------------- norm, rope --

def test_rope_frequencies():
    """exp2 and the products are within a few last places of fp64."""
    for R, base in ((64, 1e7), (2, 1e4), (256, 5e5), (20, 1e7)):
        i = np.arange(R // 2)
        f = base ** (-2 * i / R)
        got = f64(gdn.gdn_rope_inv_freq(R, base))
        assert np.all(np.abs(got - f) <= 2.0 ** -47 * f)
        got = f64(gdn.gdn_rope_inv_freq(R, base, factor=8.0))
        assert np.all(np.abs(got - f / 8) <= 2.0 ** -47 * f)
        got = f64(gdn.gdn_rope_inv_freq(R, base, factor=8.0, context=8192))
        keep = np.clip((8192 * f / (2 * np.pi) - 1) / 31, 0, 1)
        assert np.all(np.abs(got - f * (keep + (1 - keep) / 8)) <= 2.0 ** -40 * f)
    assert gdn.gdn_rope_inv_freq(0).numel() == 0


def cache(pages, page, H, D, dtype, heads_first, fill=None):
    shape = (pages, H, page, D) if heads_first else (pages, page, H, D)
    t = torch.randn(shape, device=DEV).to(dtype) if fill is None else torch.full(
        shape, fill, dtype=dtype, device=DEV)
    return t.transpose(1, 2) if heads_first else t


def check_norm_rope(T, H_q, H_kv, D, R, *, x_dtype=BF16, dtype=F16, interleaved=False, axes=3,
                    norm="both", w_dtype=BF16, page=16, heads_first=False, scale=1.0, pad=(),
                    far=0, slots="map", scatter=None, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1000 * T)
    rows = torch.randn((T, (H_q + 2 * H_kv) * D + 16), generator=g, device=DEV).to(x_dtype)
    q, k, v = (a.unflatten(1, (-1, D)) for a in
               rows[:, :-16].split([H_q * D, H_kv * D, H_kv * D], dim=1))
    pages = -(-max(T, 1) // page) + 2
    kc, vc = (cache(pages, page, H_kv, D, dtype, heads_first) for _ in range(2))
    kc0, vc0 = f64(kc), f64(vc)
    slot = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32)
    for t, s in pad:
        slot[t] = s if s < 0 else pages * page + s
    if slots != "map":
        slot = torch.arange(T, dtype=torch.int32, device=DEV)
    pos = torch.randint(0, 1 + abs(far) + T, (axes, T), generator=g, device=DEV).to(torch.int32)
    if far < 0:
        pos = -pos
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(w_dtype)
              if norm in ("both", side) else None for side in "qk")
    inv = gdn.gdn_rope_inv_freq(R, 1e7) if R else None
    q_out = torch.full((T, H_q, D), 3.0, dtype=dtype, device=DEV)
    got = gdn.gdn_qk_norm_rope(
        q, k, v, kc, vc, slot_map=slot if slots == "map" else None, q_norm_w=wq, k_norm_w=wk,
        positions=(pos if axes == 3 else pos[0]) if R else None, inv_freq=inv,
        interleaved=interleaved, rope_scale=scale, q_out=q_out)
    assert got is q_out
    s = slot.tolist()
    live = [t for t in range(T) if 0 <= s[t] < pages * page]
    fr = f64(inv) if R else None
    for name, x, w in (("q", q, wq), ("k", k, wk)):
        y, size = ref.norm_rope(f64(x), None if w is None else f64(w), f64(pos), fr, interleaved,
                                scale)
        tol = ref.norm_rope_bound(y, size, D, dtype)
        if name == "q":
            want = np.full((T, H_q, D), 3.0)
            want[live] = y[live]
            assert np.all(np.abs(f64(q_out) - want)[live] <= tol[live])
            dead = [t for t in range(T) if t not in set(live)]
            assert np.all(f64(q_out)[dead] == 3.0)
        else:
            d = f64(kc)
            for t in live:
                p, o = divmod(s[t], page)
                assert np.all(np.abs(d[p, o] - y[t]) <= tol[t]), t
                d[p, o] = kc0[p, o]
            assert np.array_equal(d, kc0)          # every other row as it was
    d, vr = f64(vc), f64(v.to(dtype))
    for t in live:
        p, o = divmod(s[t], page)
        assert np.array_equal(d[p, o], vr[t])
        d[p, o] = vc0[p, o]
    assert np.array_equal(d, vc0)


@pytest.mark.parametrize("D,R", [(256, 64), (256, 256), (256, 20), (128, 128), (128, 34), (64, 64),
                                 (64, 2), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_dims(D, R, interleaved):
    for T in (1, 3, 130):
        check_norm_rope(T, 6, 2, D, R, interleaved=interleaved, page=7)


@pytest.mark.parametrize("x_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_rope_types(x_dtype, dtype):
    for w_dtype in (BF16, F16, F32):
        check_norm_rope(21, 3, 1, 128, 32, x_dtype=x_dtype, dtype=dtype, w_dtype=w_dtype, axes=1)


@pytest.mark.parametrize("norm", ["q", "k", "none"])
def test_norm_rope_one_side_normed(norm):
    check_norm_rope(9, 4, 4, 64, 16, norm=norm, axes=1, scale=1.2079)


def test_norm_rope_layouts_padding_and_far_positions():
    check_norm_rope(700, 24, 4, 256, 64, far=250000)                # several tokens per block
    check_norm_rope(2001, 8, 2, 128, 128, dtype=BF16, heads_first=True, interleaved=True,
                    axes=1, pad=[(0, -1), (5, 0), (1999, -2 ** 31), (2000, 7)])
    check_norm_rope(50, 2, 2, 64, 64, far=2 ** 31 - 200, page=1)
    check_norm_rope(50, 2, 2, 64, 64, far=-2 ** 20 - 50, page=64)
    check_norm_rope(64, 2, 1, 64, 64, slots="none", page=32)
    check_norm_rope(5, 16, 16, 256, 96, heads_first=True, page=3)


def test_norm_rope_parts_of_the_call():
    """Queries alone, keys and values alone (a plain append), in place, no tokens."""
    T, H, D = 33, 4, 128
    x = torch.randn(T, H, D, device=DEV).half()
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv = gdn.gdn_rope_inv_freq(D, 1e4)
    w = torch.ones(D, device=DEV)
    alone = gdn.gdn_qk_norm_rope(x, None, None, q_norm_w=w, positions=pos, inv_freq=inv)
    y, size = ref.norm_rope(f64(x), f64(w), f64(pos)[None], f64(inv), False, 1.0)
    assert np.all(np.abs(f64(alone) - y) <= ref.norm_rope_bound(y, size, D, F16))
    inplace = x.clone()
    gdn.gdn_qk_norm_rope(inplace, None, None, q_norm_w=w, positions=pos, inv_freq=inv,
                         q_out=inplace)
    assert torch.equal(inplace, alone)
    skip = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    skip[4] = 0
    kept = x.clone()
    gdn.gdn_qk_norm_rope(kept, None, None, slot_map=skip, q_norm_w=w, positions=pos, inv_freq=inv,
                         q_out=kept)
    x[4] = alone[4]
    assert torch.equal(kept, x)
    kc, vc = (torch.zeros(3, 16, H, D, dtype=F16, device=DEV) for _ in range(2))
    slots = torch.randperm(48, device=DEV)[:T].to(torch.int32)
    assert gdn.gdn_qk_norm_rope(None, x, alone, kc, vc, slot_map=slots) is None
    assert torch.equal(kc.flatten(0, 1)[slots.long()], x)
    assert torch.equal(vc.flatten(0, 1)[slots.long()], alone)
    assert int((kc != 0).any(-1).any(-1).sum()) == T
    assert gdn.gdn_qk_norm_rope(x[:0], None, None).shape == (0, H, D)


def test_norm_rope_extreme_values():
    """Values past fp16's range saturate, NaN stays, a zero row stays zero."""
    D = 64
    x = torch.zeros(4, 1, D, device=DEV)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = 1e6, -1e30, float("inf")
    x[1, 0, 3] = float("nan")
    kc, vc = (torch.zeros(1, 4, 1, D, dtype=F16, device=DEV) for _ in range(2))
    gdn.gdn_qk_norm_rope(None, x, x, kc, vc, k_norm_w=torch.ones(D, device=DEV))
    v = vc[0, :, 0]
    assert v[0, :3].tolist() == [65504.0, -65504.0, 65504.0]
    assert bool(v[1, 3].isnan()) and bool((v[2:] == 0).all())
    assert bool(kc[0, 1].isnan().all()) and bool((kc[0, 2:] == 0).all())


# --------------------------------------------------------------- paged attention --

def decode_state(lens, H_q, H_kv, D, page, dtype, heads_first=False, gate=True, seed=0, spare=2):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    N = len(lens)
    held = [-(-n // page) for n in lens]
    width = max(1, max(held))
    P = sum(held) + spare
    ids = torch.randperm(P, generator=g, device=DEV).tolist()
    table = torch.full((N, width), -3, dtype=torch.int32)
    kc, vc = (cache(P, page, H_kv, D, dtype, heads_first) for _ in range(2))
    at = 0
    for n, h in enumerate(held):
        table[n, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
        at += h
        if lens[n] % page:                       # rows behind the end were never written
            kc[ids[at - 1], lens[n] % page:] = float("nan")
            vc[ids[at - 1], lens[n] % page:] = float("inf")
    for i in ids[at:]:
        kc[i], vc[i] = float("nan"), float("nan")
    q = torch.randn((N, H_q, D), generator=g, device=DEV).to(dtype)
    gt = torch.randn((N, H_q, D), generator=g, device=DEV).to(BF16) if gate else None
    return dict(q=q, kc=kc, vc=vc, table=table.to(DEV), lens=i32(lens).reshape(-1), gate=gt)


def run_decode(s, **kw):
    return gdn.gdn_paged_attention_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                          gate=s["gate"], **kw)


def check_decode(s, o, lse=None, scale=None, only=None):
    N, H_q, D = s["q"].shape
    page, H_kv = s["kc"].shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    lens = s["lens"].tolist()
    got = f64(o)
    for n in range(N) if only is None else only:
        pages = s["table"][n, :-(-lens[n] // page)].long()
        k, v = (f64(c[pages].reshape(-1, H_kv, D)[:lens[n]]) for c in (s["kc"], s["vc"]))
        r, l, err, lerr = ref.decode(f64(s["q"][n]), k, v, scale,
                                     None if s["gate"] is None else f64(s["gate"][n]))
        tol = ref.HALF[o.dtype] * np.abs(r) + ref.TINY[o.dtype] + err
        d = np.abs(got[n] - r)
        assert np.all(d <= tol), (n, lens[n], float((d - tol).max()))
        if lse is not None:
            gl = f64(lse[n])
            same = gl == l
            assert np.all(np.abs(gl[~same] - l[~same]) <= lerr[~same]), (n, lens[n])


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 130, 500, 0, 1029]


@pytest.mark.parametrize("D", [256, 128, 64])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H_q,H_kv", [(6, 1), (8, 8), (12, 4), (16, 2), (16, 1), (11, 1)])
def test_decode_heads_types(D, dtype, H_q, H_kv):
    s = decode_state(LENS, H_q, H_kv, D, 16, dtype, seed=D + H_q)
    lse = torch.empty(len(LENS), H_q, device=DEV)
    check_decode(s, run_decode(s, lse=lse, o_dtype=F32), lse)


@pytest.mark.parametrize("page", [1, 7, 48, 64, 300])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("o_dtype", [BF16, F16, F32])
def test_decode_pages_layouts_outputs(page, heads_first, o_dtype):
    s = decode_state(LENS + [301, 2000], 8, 2, 128, page, BF16, heads_first,
                     gate=o_dtype != F16, seed=page)
    check_decode(s, run_decode(s, o_dtype=o_dtype))


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [40000], [9000, 1, 0, 9001], [1] * 700,
                                  [0] * 333 + [70] + [0] * 100 + [5, 0], [64] * 150])
def test_decode_splits(lens):
    """One long sequence over all CTAs, many short ones, runs of empty ones."""
    s = decode_state(lens, 24, 4, 256, 64, F16, seed=len(lens))
    lse = torch.empty(len(lens), 24, device=DEV)
    o = run_decode(s, lse=lse)
    some = list(range(len(lens)))[:: max(1, len(lens) // 40)]
    some += [n for n, x in enumerate(lens) if x not in (0, lens[0])][:20]
    check_decode(s, o, lse, only=some)
    again = run_decode(s)
    assert torch.equal(o, again)                 # the same bits whatever runs first


@pytest.mark.parametrize("D,H_q,H_kv,N,lo,hi", [
    (256, 8, 4, 40, 3900, 4300), (256, 24, 4, 700, 0, 1100), (256, 32, 2, 80, 3000, 5000),
    (128, 8, 4, 70, 4500, 4900), (128, 16, 1, 300, 4100, 4300), (64, 16, 16, 61, 2500, 2900),
    (64, 16, 1, 150, 8100, 8300)])
def test_decode_taken_over_ranges(D, H_q, H_kv, N, lo, hi):
    """Enough work that CTAs which are done take over ranges that have not started;
    more sequences than are summed singly; all of them over the same few pages."""
    rng = np.random.default_rng([D, H_q, N])
    lens = rng.integers(lo, hi + 1, N).tolist()
    page, dtype = 16, F16
    width = -(-hi // page)
    P = width + 7
    kc, vc = (cache(P, page, H_kv, D, dtype, D == 128) for _ in range(2))
    table = torch.stack([torch.randperm(P, device=DEV)[:width] for _ in range(N)]).to(torch.int32)
    s = dict(q=torch.randn(N, H_q, D, device=DEV).to(dtype), kc=kc, vc=vc, table=table,
             lens=i32(lens), gate=torch.randn(N, H_q, D, device=DEV).bfloat16())
    ws = torch.empty(gdn.gdn_paged_attention_decode_workspace(H_q, H_kv, D), dtype=torch.uint8,
                     device=DEV)
    lse = torch.empty(N, H_q, device=DEV)
    o = run_decode(s, lse=lse, workspace=ws)
    assert gdn.gdn_attention_status(ws) == 0
    check_decode(s, o, lse, only=sorted(rng.choice(N, min(N, 12), replace=False).tolist()))
    # no row is missed: the same sequences in calls too small for any taking over
    for a in range(0, N, 16):
        part = {k: v[a:a + 16] if k in ("q", "table", "lens", "gate") else v for k, v in s.items()}
        d = (run_decode(part, o_dtype=F32) - o[a:a + 16].float()).abs()
        assert float((d / (1e-4 + o[a:a + 16].float().abs())).max()) < 2.0 ** -7
    for _ in range(4):
        assert torch.equal(run_decode(s, workspace=ws), o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run_decode(s, workspace=ws)
    for _ in range(2):
        again.zero_()
        graph.replay()
        assert torch.equal(again, o)
    table[1, 0] = P                              # a bad page there, and a bad length
    s["lens"][2] = width * page + 1
    b = run_decode(s, workspace=ws)
    assert gdn.gdn_attention_status(ws) == -1
    bad = torch.tensor([lens[1] > 0 and n == 1 or n == 2 for n in range(N)], device=DEV)
    assert bool(b[bad].isnan().all()) and bool(b[~bad].isfinite().all())


def test_decode_most_sequences():
    """65535 sequences, nearly all empty; the last one long."""
    N, D = 65535, 64
    s = decode_state([33, 0, 700], 2, 1, D, 16, BF16, gate=False, seed=3)
    at = [5, 30000, N - 1]
    lens = torch.zeros(N, dtype=torch.int32, device=DEV)
    table = torch.full((N, s["table"].shape[1]), -1, dtype=torch.int32, device=DEV)
    q = torch.randn(N, 2, D, device=DEV).bfloat16()
    lens[at], table[at], q[at] = s["lens"], s["table"], s["q"]
    o = run_decode(dict(s, q=q, lens=lens, table=table))
    check_decode(s, o[at])
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not bool(o[rest].any())


def test_calls_at_the_same_time():
    """Two host threads on two streams, each with its own buffers."""
    import threading
    states = [decode_state([1500, 40, 900, 7] * 4, 12, 2, 128, 16, BF16, seed=20 + i)
              for i in range(2)]
    want = [run_decode(s) for s in states]
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                if not torch.equal(run_decode(states[i]), want[i]):
                    bad.append(i)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_decode_peaked_and_flat_scores():
    """Scores of hundreds (one key takes all), keys of zero (the mean of the values),
    a scale of its own, a score of -inf and infinite values."""
    s = decode_state([100, 1000, 65, 3], 4, 2, 64, 16, BF16, gate=False, seed=4)
    s["kc"].mul_(40)
    check_decode(s, run_decode(s, o_dtype=F32, scale=0.5), scale=0.5)
    s["kc"].nan_to_num_(0).zero_()
    check_decode(s, run_decode(s, o_dtype=F32))
    s = decode_state([40], 2, 1, 64, 8, F16, gate=False, seed=5)
    s["q"].abs_()
    first = int(s["table"][0, 0])
    s["kc"][first] = float("-inf")               # the first eight keys: weight 0
    o = run_decode(s, o_dtype=F32)
    rest = dict(s, table=s["table"][:, 1:].contiguous(), lens=i32([32]))
    check_decode(rest, o)
    s["vc"][first, 3, 0, 5] = float("inf")       # 0 * inf of a live key is NaN, in its dim alone
    o = run_decode(s, o_dtype=F32)
    assert bool(o[0, :, 5].isnan().all()) and int(o.isnan().sum()) == 2


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("above", [10.0, 14.0, 17.0])
def test_decode_one_key_above_many(dtype, above):
    """One key takes most of the sum and 60000 equal ones share the rest, each with a
    weight of e^-above of the first's: their common rounding must not add up. 150
    such sequences over the same pages, so that none is cut into many pieces."""
    L, D, page = 60001, 64, 64
    s = decode_state([L, L], 2, 1, D, page, dtype, gate=False, seed=6)
    s["q"].fill_(1.0)
    for at in (0, L - 1):                        # the key comes first, or last
        for n in range(2):
            pages = s["table"][n].long()
            s["kc"][pages] = torch.where(s["kc"][pages].isnan(), s["kc"][pages], 0.0)
            s["vc"][pages] = torch.where(s["vc"][pages].isinf(), s["vc"][pages],
                                         1 + 0.1 * s["vc"][pages].clamp(-3, 3))
            s["kc"][pages[at // page], at % page] = above * D ** 0.5 / D
            s["vc"][pages[at // page], at % page] = -1.0
        many = dict(s, **{k: s[k].repeat(75, *[1] * (s[k].dim() - 1)) for k in ("q", "table", "lens")})
        lse = torch.empty(150, 2, device=DEV)
        check_decode(many, run_decode(many, o_dtype=F32, lse=lse), lse, only=[0, 75, 149])


def test_decode_views_shared_pages_and_workspace():
    """q and gate as views, sequences that share pages, k and v in one buffer, one
    workspace for calls of different shapes, contents of it before a call."""
    N, H_q, H_kv, D, page = 5, 8, 2, 128, 16
    s = decode_state([200, 64, 33, 1, 129], H_q, H_kv, D, page, F16, seed=8)
    both = torch.empty(s["kc"].shape[0], 2, page, H_kv, D, dtype=F16, device=DEV)
    both[:, 0], both[:, 1] = s["kc"], s["vc"]
    wide = torch.randn(N, 3 * H_q, D, device=DEV).half()
    gate = torch.randn(N, 3 * H_q, D, device=DEV).bfloat16()
    table = torch.full((N, 40), -1, dtype=torch.int32, device=DEV)
    view = table[:, 5:5 + s["table"].shape[1]]
    view.copy_(s["table"])
    view[1, :4] = view[0, :4]                    # a shared prefix
    s = dict(s, q=wide[:, 5:5 + H_q], gate=gate[:, H_q:2 * H_q], kc=both[:, 0], vc=both[:, 1],
             table=view)
    need = max(gdn.gdn_paged_attention_decode_workspace(H_q, H_kv, D),
               gdn.gdn_paged_attention_decode_workspace(24, 4, 256))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    check_decode(s, run_decode(s, workspace=ws))
    assert gdn.gdn_attention_status(ws) == 0
    t = decode_state([3000, 2], 24, 4, 256, 64, F16, seed=9)
    check_decode(t, run_decode(t, workspace=ws))
    check_decode(s, run_decode(s, workspace=ws))


@pytest.mark.parametrize("page", [8, 16, 64, 192])
@pytest.mark.parametrize("D", [64, 256])
def test_decode_cache_strides(page, D):
    """Padded pages, tokens and heads (strides that are no multiples of one another),
    heads cut out of wider rows, one head, one page, in the order given and turned."""
    lens = [3 * page + 5, page, 1, 2 * page - 1]
    for H_kv, pad in ((2, (24, 0, 0)), (2, (0, 8, 0)), (3, (0, 0, 64)), (1, (0, 0, 0)),
                      (1, (8, 64, 0))):
        for heads_first in (False, True):
            s = decode_state(lens, 4 * H_kv, H_kv, D, page, BF16, heads_first, seed=page + H_kv)
            for name in ("kc", "vc"):
                c = s[name].transpose(1, 2) if heads_first else s[name]
                P, a, b, _ = c.shape
                inner = D + pad[2]
                rows = b * inner + pad[1]
                wide = torch.full((P, a * rows + pad[0]), float("nan"), dtype=BF16, device=DEV)
                view = wide.as_strided((P, a, b, D), (a * rows + pad[0], rows, inner, 1))
                view.copy_(c)
                s[name] = view.transpose(1, 2) if heads_first else view
            check_decode(s, run_decode(s))
    s = decode_state([page - 1], 4, 2, D, page, F16, spare=0)
    assert s["kc"].shape[0] == 1
    check_decode(s, run_decode(s))


def test_decode_bad_pages_and_lengths():
    """Named by the status, NaN in their rows, no other row touched; the next
    call on the workspace is clean. Pages are looked at on the device before any copy."""
    s = decode_state([200, 100, 50, 5000], 8, 2, 64, 16, F16, gate=False, seed=11)
    good = run_decode(s)
    ws = torch.empty(gdn.gdn_paged_attention_decode_workspace(8, 2, 64), dtype=torch.uint8,
                     device=DEV)
    bad = dict(s, table=s["table"].clone())
    bad["table"][1, 3] = s["kc"].shape[0]        # one past the last page
    bad["table"][3, 200] = -1
    lse = torch.empty(4, 8, device=DEV)
    o = run_decode(bad, workspace=ws, lse=lse)
    assert gdn.gdn_attention_status(ws) == -1
    assert torch.equal(o[[0, 2]], good[[0, 2]]) and bool(o[[1, 3]].isnan().all())
    assert bool(lse[[1, 3]].isnan().all()) and bool(lse[[0, 2]].isfinite().all())
    bad = dict(s, lens=i32([200, -1, 50, s["table"].shape[1] * 16 + 1]))
    o = run_decode(bad, workspace=ws)
    assert gdn.gdn_attention_status(ws) == -1
    assert torch.equal(o[[0, 2]], good[[0, 2]]) and bool(o[[1, 3]].isnan().all())
    assert torch.equal(run_decode(s, workspace=ws), good)
    assert gdn.gdn_attention_status(ws) == 0


def test_decode_streams_and_graphs():
    """On a stream of its own; two captured graphs on one workspace, replayed on new
    lengths and tables."""
    s = decode_state([700, 30, 0, 64], 12, 2, 128, 16, BF16, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = run_decode(s, stream=side)
    side.synchronize()
    check_decode(s, o)
    o = run_decode(s, stream=side.cuda_stream)
    side.synchronize()
    check_decode(s, o)
    ws = torch.empty(gdn.gdn_paged_attention_decode_workspace(12, 2, 128), dtype=torch.uint8,
                     device=DEV)
    outs = [torch.empty(4, 12, 128, dtype=BF16, device=DEV) for _ in range(2)]
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_decode(s, workspace=ws, o=out)
        graphs.append(g)
    for lens in ([700, 30, 0, 64], [1, 0, 0, 3], [699, 29, 0, 63]):
        s["lens"].copy_(i32(lens))
        for g, out in zip(graphs, outs):
            g.replay()
        check_decode(s, outs[0])
        assert torch.equal(*outs)


def test_decode_offsets_past_32_bits():
    """A cache of more than 2^32 elements, with the sequence's pages at its far end."""
    H_kv, D, page = 4, 256, 64
    P = (1 << 32) // (H_kv * D * page) + 5
    kc = torch.empty(P, page, H_kv, D, dtype=F16, device=DEV)
    vc = torch.empty_like(kc)
    kc[-6:], vc[-6:] = torch.randn(2, 6, page, H_kv, D, device=DEV).half()
    s = dict(q=torch.randn(2, 24, D, device=DEV).half(), kc=kc, vc=vc, gate=None,
             table=i32([[P - 1, P - 3, P - 5], [P - 2, P - 6, P - 4]]), lens=i32([190, 130]))
    check_decode(s, run_decode(s))
    rows = torch.randn(3, 4, D, device=DEV).half()
    slots = i32([(P - 1) * page + 63, (P - 2) * page, (P - 6) * page + 5])
    gdn.gdn_qk_norm_rope(None, rows, rows, kc, vc, slot_map=slots)
    for t, x in enumerate(slots.tolist()):
        assert torch.equal(kc[x // page, x % page], rows[t])
        assert torch.equal(vc[x // page, x % page], rows[t])
    check_decode(s, run_decode(s))


# -------------------------------------------------------------- a server's steps --

def test_serving_steps_against_the_oracle():
    """Prompts through gdn_attention_prefill, their rows appended to pages that
    gdn_page_plan gave; then decode steps by plan, norm + rotary + append and
    paged attention, while one request ends, one starts and one is cut back: every
    row against the layer's oracle, with the attention layer's bar."""
    H_q, H_kv, D, page, P = 24, 4, 256, 16, 64
    total = 300
    seqs = [gi.attention_inputs(total, seed=20 + n) for n in range(4)]
    for s in seqs[1:]:
        s["q_norm_w"], s["k_norm_w"] = seqs[0]["q_norm_w"], seqs[0]["k_norm_w"]
    wq, wk = seqs[0]["q_norm_w"].to(DEV), seqs[0]["k_norm_w"].to(DEV)
    want_o = []
    for s in seqs:
        o, _, _ = oracle.attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), f64(s["gate"]),
                                   f64(s["q_norm_w"]), f64(s["k_norm_w"]),
                                   cu_seqlens=np.array([0, total]))
        want_o.append(o)
    kc, vc = (torch.full((P, page, H_kv, D), float("nan"), dtype=F16, device=DEV)
              for _ in range(2))
    table = torch.full((4, 20), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(P, dtype=torch.int32, device=DEV)
    lens, count = i32([0, 0, 0, 0]), i32([P])
    inv = gdn.gdn_rope_inv_freq(64, 1e7)

    def rows(name, now, then):
        return torch.cat([seqs[n][name][a:b] for n, (a, b) in enumerate(zip(now, then)) if b > a])

    def place(then):
        nonlocal lens, count
        now = lens.tolist()
        new = sum(max(0, b - a) for a, b in zip(now, then))
        p = gdn.gdn_page_plan(lens, i32(then), table, free, count, page, token_capacity=new + 3)
        assert p.info[3] == 0 and p.info[0] == new
        lens, count = p.new_lens, p.new_count
        return now, p, new

    def prompt(then):
        now, p, new = place(then)
        x = {k: rows(k, now, then).to(DEV) for k in ("q", "k", "v", "gate")}
        o, k_rot, v_h = gdn.gdn_attention_prefill(x["q"], x["k"], x["v"], x["gate"], wq, wk,
                                                  p.cu_new)
        gdn.gdn_qk_norm_rope(None, k_rot, v_h, kc, vc, slot_map=p.slot_map[:new])
        return o

    def bar(got, r):
        rms = np.sqrt(np.mean(r ** 2, axis=-1, keepdims=True))
        assert np.all(np.abs(got - r) <= 2.0 ** -8 * np.abs(r) + 1e-2 * rms)

    def step(then):
        now, p, new = place(then)
        live = [n for n in range(4) if then[n] > now[n]]
        x = {k: rows(k, now, then).to(DEV) for k in ("q", "k", "v", "gate")}
        pos = p.positions[:new]
        q = gdn.gdn_qk_norm_rope(x["q"], x["k"], x["v"], kc, vc, slot_map=p.slot_map[:new],
                                 q_norm_w=wq, k_norm_w=wk, positions=pos, inv_freq=inv)
        at = torch.tensor(live, device=DEV)
        o = gdn.gdn_paged_attention_decode(q, kc, vc, table[at], lens[at], gate=x["gate"])
        for i, n in enumerate(live):
            bar(f64(o[i]), want_o[n][now[n]])

    o = prompt([100, 63, 16, 0])
    at = 0
    for n, length in enumerate([100, 63, 16]):
        bar(f64(o[at:at + length]), want_o[n][:length])
        at += length
    step([101, 64, 17, 0])
    step([102, 65, 18, 0])
    step([0, 66, 19, 0])                         # the first ends
    prompt([0, 66, 19, 290])                     # another starts on its pages
    for _ in range(3):
        step([0] + [n + 1 for n in lens.tolist()[1:]])
    place([0, 65, 22, 293])                      # the second is cut back and goes on
    step([0, 66, 22, 294])
    held = sum(-(-n // page) for n in lens.tolist())
    assert int(count) == P - held
    mine = [table[n, :-(-x // page)].tolist() for n, x in enumerate(lens.tolist())]
    assert sorted(sum(mine, []) + free[:int(count)].tolist()) == list(range(P))
    assert math.isfinite(float(count))


def test_captured_step_equals_eager_steps():
    """A whole decode step (plan, norm + rotary + append, attention, the copies that adopt
    the plan) captured once and replayed, with a request that never grows; bit for bit
    the same as the eager calls."""
    H_q, H_kv, D, page, P, N = 12, 2, 128, 16, 40, 5
    inv = gdn.gdn_rope_inv_freq(64, 1e6, factor=4.0, context=256)
    w = torch.randn(D, device=DEV)
    steps = [[torch.randn(N, H, D, device=DEV).bfloat16() for H in (H_q, H_kv, H_kv)]
             for _ in range(40)]

    class Server:
        def __init__(self):
            self.kc, self.vc = (torch.zeros(P, H_kv, page, D, dtype=BF16, device=DEV).transpose(1, 2)
                                for _ in range(2))
            self.table = torch.full((N, 20), -1, dtype=torch.int32, device=DEV)
            self.free = torch.arange(P, dtype=torch.int32, device=DEV).flip(0).contiguous()
            self.lens, self.count = i32([0] * N), i32([P])
            self.grow = i32([1, 1, 0, 1, 1])
            self.x = [t.clone() for t in steps[0]]
            self.ws = torch.empty(gdn.gdn_paged_attention_decode_workspace(H_q, H_kv, D),
                                  dtype=torch.uint8, device=DEV)

        def step(self):
            p = gdn.gdn_page_plan(self.lens, self.lens + self.grow, self.table, self.free,
                                  self.count, page, token_capacity=N)
            # rows of the requests that got a token, in order, padding behind
            row = torch.searchsorted(p.cu_new, torch.arange(N, device=DEV, dtype=torch.int32),
                                     right=True, out_int32=True) - 1
            q, k, v = (t[row.clamp(max=N - 1)] for t in self.x)
            q = gdn.gdn_qk_norm_rope(q, k, v, self.kc, self.vc, slot_map=p.slot_map, k_norm_w=w,
                                     q_norm_w=w, positions=p.positions, inv_freq=inv)
            back = torch.zeros(N, H_q, D, dtype=BF16, device=DEV)
            back[row.clamp(max=N - 1).long()] = q      # rows of padding end up in the last
            self.o = gdn.gdn_paged_attention_decode(back, self.kc, self.vc, self.table,
                                                    p.new_lens * self.grow, workspace=self.ws)
            self.lens.copy_(p.new_lens)
            self.count.copy_(p.new_count)
            return self.o

    eager, captured = Server(), Server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Server().step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.step()
    for xs in steps:
        for s in (eager, captured):
            for a, b in zip(s.x, xs):
                a.copy_(b)
        o = eager.step()
        graph.replay()
        n = 4                                          # the last row may hold padding's queries
        assert torch.equal(out[:n], o[:n])
        for name in ("lens", "count", "table", "free", "kc", "vc"):
            assert torch.equal(getattr(eager, name), getattr(captured, name)), name
    assert eager.lens.tolist() == [40, 40, 0, 40, 40] and int(eager.count) == P - 12
    assert not bool(eager.o[2].any())
