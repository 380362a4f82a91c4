"""CPU: refusals of the paged-cache entry points, by the C ABI (nothing is
launched: the pointers are never followed) and by the Python binding."""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn
from gated_delta_rule_106_b200 import _build
import _paged as ref

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
BF16, F32, F16 = 0, 1, 2
A = 1 << 40                        # an aligned address that nothing follows
STEP = 1 << 34                     # apart from one another


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def plan(lib, **kw):
    a = dict(lens=A, want=A + STEP, N=4, table=A + 2 * STEP, row=8, width=8, free=A + 3 * STEP,
             count=A + 4 * STEP, P=64, page=16, cap=32, new_lens=A + 5 * STEP, cu=A + 6 * STEP,
             slots=A + 7 * STEP, pos=A + 8 * STEP, new_count=A + 9 * STEP, info=A + 10 * STEP,
             s=None)
    a.update(kw)
    return lib.gdn_page_plan(*a.values())


def test_plan_validation(lib):
    for kw in (dict(N=-1), dict(width=0), dict(P=0), dict(page=0), dict(cap=-1),
               dict(cap=(1 << 30) + 1), dict(row=7), dict(P=1 << 28, page=16),
               dict(width=1 << 28, row=1 << 28, page=16), dict(width=1 << 20, row=1 << 20, N=4096),
               dict(free=None), dict(count=None), dict(cu=None), dict(new_count=None),
               dict(slots=None), dict(lens=None), dict(want=None), dict(table=None),
               dict(new_lens=None)):
        assert plan(lib, **kw) == INVALID, kw
    assert plan(lib, N=16385) == UNSUPPORTED
    for kw in (dict(lens=A + 2), dict(table=A + 2 * STEP + 1), dict(slots=A + 7 * STEP + 4),
               dict(pos=A + 8 * STEP + 8), dict(info=A + 10 * STEP + 2)):
        assert plan(lib, **kw) == MISALIGNED, kw
    # outputs must not lie over inputs or one another
    for kw in (dict(new_lens=A), dict(new_lens=A + STEP + 12), dict(new_count=A + 4 * STEP),
               dict(slots=A), dict(pos=A + 7 * STEP), dict(cu=A + 5 * STEP),
               dict(info=A + 9 * STEP), dict(free=A + 4 * STEP), dict(table=A),
               dict(new_lens=A + 2 * STEP + 4 * 31)):
        assert plan(lib, **kw) == INVALID, kw


def test_rope_validation(lib):
    call = lambda R=64, base=1e7, f=1.0, ctx=0.0, hi=32.0, lo=1.0, out=A: (  # noqa: E731
        lib.gdn_rope_inv_freq(R, base, f, ctx, hi, lo, out, None))
    nan = float("nan")
    assert call(R=3) == call(R=-2) == call(R=258) == UNSUPPORTED
    assert call(base=1.0) == call(base=nan) == call(f=0.5) == call(f=nan) == INVALID
    assert call(ctx=-1.0) == call(ctx=1.0, hi=1.0) == call(out=None) == INVALID
    assert call(out=A + 4) == MISALIGNED
    assert call(R=0, out=None) == OK


def rope(lib, **kw):
    a = dict(q=A, qs=24 * 256, k=A + STEP, ks=1024, v=A + 2 * STEP, vs=1024, xd=BF16, wq=A, wk=A,
             wd=F32, eps=1e-6, pos=A, axes=3, inv=A, R=64, inter=0, rs=1.0, slots=A, T=8, Hq=24,
             Hkv=4, D=256, qo=A + 3 * STEP, kc=A + 4 * STEP, kp=16384, kt=1024, kh=256,
             vc=A + 5 * STEP, vp=16384, vt=1024, vh=256, P=8, page=16, od=F16, s=None)
    a.update(kw)
    return lib.gdn_qk_norm_rope(*a.values())


def test_norm_rope_validation(lib):
    for kw in (dict(D=96), dict(R=63), dict(R=258), dict(D=64, R=66), dict(od=F32), dict(od=9)):
        assert rope(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(xd=3), dict(wd=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(T=-1),
               dict(T=(1 << 30) + 1), dict(q=None, k=None, v=None), dict(k=None), dict(v=None),
               dict(Hq=0), dict(Hkv=0), dict(axes=2), dict(qs=24 * 256 - 8), dict(ks=1016),
               dict(vs=0), dict(kc=None), dict(vc=None), dict(P=0), dict(page=0),
               dict(P=1 << 28), dict(kp=-1024), dict(kt=128), dict(vh=0), dict(qo=None),
               dict(pos=None), dict(inv=None), dict(slots=None, T=129),
               # over its inputs, but not in place
               dict(qo=A), dict(qo=A + 16, qs=24 * 256, xd=F16), dict(qo=A + STEP),
               dict(qo=A + 2 * STEP + 4096)):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(qs=24 * 256 + 4), dict(q=A + 8), dict(k=A + STEP + 2), dict(qo=A + 3 * STEP + 8),
               dict(kc=A + 4 * STEP + 8), dict(kp=16388), dict(vt=1028), dict(vh=260),
               dict(wq=A + 2), dict(inv=A + 4), dict(pos=A + 2), dict(slots=A + 1),
               dict(xd=F32, qs=24 * 256 + 2)):
        assert rope(lib, **kw) == MISALIGNED, kw
    assert rope(lib, T=0) == OK


def decode(lib, **kw):
    a = dict(q=A, qs=24 * 256, kc=A, kp=65536, kt=1024, kh=256, vc=A, vp=65536, vt=1024, vh=256,
             kd=F16, P=64, page=64, table=A, row=16, width=16, lens=A, gate=None, gs=0, N=4, Hq=24,
             Hkv=4, D=256, scale=0.0625, o=A + STEP, od=BF16, lse=None, ws=A, wb=1 << 40, s=None)
    a.update(kw)
    return lib.gdn_paged_attention_decode(*a.values())


def test_decode_validation(lib):
    for kw in (dict(D=80), dict(kd=F32), dict(Hq=68, qs=68 * 256)):
        assert decode(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(Hq=25), dict(Hkv=0), dict(N=-1), dict(N=65536), dict(od=5),
               dict(scale=float("nan")), dict(qs=24 * 256 - 8), dict(gate=A, gs=256),
               dict(width=0), dict(row=15), dict(width=1 << 26, row=1 << 26), dict(kc=None),
               dict(P=0), dict(page=0), dict(kt=0), dict(kh=64), dict(P=1 << 26), dict(q=None),
               dict(table=None), dict(lens=None), dict(o=None), dict(ws=None),
               dict(wb=lib.gdn_paged_attention_decode_workspace(24, 4, 256) - 1)):
        assert decode(lib, **kw) == INVALID, kw
    for kw in (dict(q=A + 2), dict(qs=24 * 256 + 4), dict(kc=A + 8), dict(vp=65540), dict(o=A + STEP + 8),
               dict(ws=A + 4), dict(gate=A + 8, gs=24 * 256), dict(gate=A, gs=24 * 256 + 1),
               dict(table=A + 2), dict(lens=A + 1), dict(lse=A + 2)):
        assert decode(lib, **kw) == MISALIGNED, kw
    # the output over the queries or the gate; more work than is counted
    for kw in (dict(o=A), dict(o=A + 4 * 24 * 512 - 16), dict(gate=A + STEP, gs=24 * 256)):
        assert decode(lib, **kw) == INVALID, kw
    assert decode(lib, N=65535, Hq=65535, Hkv=65535, qs=65535 * 256, width=1 << 25, row=1 << 25,
                  kp=65535 * 256 * 64, kt=65535 * 256) == UNSUPPORTED
    assert decode(lib, N=0) == OK
    assert lib.gdn_paged_attention_decode_workspace(24, 5, 256) == 0
    assert lib.gdn_paged_attention_decode_workspace(24, 4, 96) == 0


def test_older_entry_points_refuse_fp16_codes(lib):
    assert lib.gdn_gated_rmsnorm(A, F16, A, BF16, A, F32, 4, 128, 1e-6, A, BF16, None) == INVALID


def given(kw, *defaults):
    """The named arguments taken out of kw, else their defaults; then the rest of kw."""
    return [kw.pop(name, value) for name, value in defaults], kw


def test_binding_checks(lib):
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    def p(**kw):
        args, kw = given(kw, ("lens", i(3)), ("want", i(3)), ("table", i(3, 4)), ("free", i(9)),
                         ("count", i(1)))
        return gdn.gdn_page_plan(*args, 16, **{"token_capacity": 8, **kw})

    for match, kw in (("want: shape", dict(want=i(2))), ("lens: dtype", dict(lens=i(3).long())),
                      ("block_table: shape", dict(table=i(2, 4))),
                      ("block_table: dtype", dict(table=i(3, 4).long())),
                      ("block_table: rows", dict(table=i(4, 3).T)),
                      ("free_count: shape", dict(count=i(2))), ("new_lens: shape", dict(new_lens=i(4))),
                      ("slot_map's length", dict(slot_map=i(7))), ("info: shape", dict(info=i(3))),
                      ("token_capacity or", dict(token_capacity=None)),
                      ("CUDA tensors only", {})):
        with pytest.raises(ValueError, match=match):
            p(**kw)
    q, k = torch.zeros(5, 8, 64).half(), torch.zeros(5, 2, 64).half()
    c = torch.zeros(3, 16, 2, 64).half()
    f, pos = torch.zeros(16, dtype=torch.float64), i(5)

    def r(**kw):
        args, kw = given(kw, ("q", q), ("k", k), ("v", k), ("kc", c), ("vc", c))
        return gdn.gdn_qk_norm_rope(*args, **kw)

    for match, kw in (("give q", dict(q=None, k=None, v=None, kc=None, vc=None)),
                      ("give q", dict(v=None)), ("give q", dict(kc=None)),
                      ("k: dtype", dict(k=k.float())), ("v: shape", dict(v=q)),
                      ("k_cache: shape", dict(kc=torch.zeros(3, 2, 16, 64).half())),
                      ("v_cache: dtype", dict(vc=c.bfloat16())),
                      ("k_cache: each row", dict(kc=torch.zeros(3, 16, 64, 2).half().transpose(2, 3))),
                      ("bf16 or fp16", dict(kc=c.float(), vc=c.float())),
                      ("out_dtype", dict(out_dtype=torch.bfloat16)),
                      ("q_out: dtype", dict(q_out=q.float())), ("q_out without", dict(q=None, q_out=q)),
                      ("slot_map: dtype", dict(slot_map=pos.long())),
                      ("k_norm_w: dtype", dict(q_norm_w=torch.ones(64).half(), k_norm_w=torch.ones(64))),
                      ("q_norm_w: shape", dict(q_norm_w=torch.ones(32))),
                      ("inv_freq: dtype", dict(inv_freq=f.float(), positions=pos)),
                      ("needs positions", dict(inv_freq=f)), ("without inv_freq", dict(positions=pos)),
                      ("positions: shape", dict(inv_freq=f, positions=i(2, 5))),
                      ("contiguous", dict(q=torch.zeros(5, 64, 8).half().transpose(1, 2))),
                      ("CUDA tensors only", {})):
        with pytest.raises(ValueError, match=match):
            r(**kw)

    def a(**kw):
        args, kw = given(kw, ("q", q), ("kc", c), ("vc", c), ("table", i(5, 2)), ("lens", i(5)))
        return gdn.gdn_paged_attention_decode(*args, **kw)

    for match, kw in (("q: dtype", dict(q=q.bfloat16())),
                      ("head dim", dict(q=torch.zeros(5, 8, 128).half(),
                                        vc=torch.zeros(3, 16, 2, 128).half())),
                      ("v_cache: shape", dict(vc=c[:2])), ("caches are", dict(kc=c.float())),
                      ("block_table: shape", dict(table=i(4, 2))),
                      ("kv_lens: dtype", dict(lens=i(5).long())),
                      ("gate: dtype", dict(gate=q)), ("gate: shape", dict(gate=q[:, :4].bfloat16())),
                      ("o: shape", dict(o=k)), ("o: dtype", dict(o=q, o_dtype=torch.float32)),
                      ("lse: shape", dict(lse=torch.zeros(8, 5))), ("CUDA tensors only", {})):
        with pytest.raises(ValueError, match=match):
            a(**kw)
    with pytest.raises(TypeError, match="unsupported dtype"):
        a(o_dtype=torch.float64)
    with pytest.raises(ValueError, match="out: shape"):
        gdn.gdn_rope_inv_freq(64, out=f)


def test_plain_plan_form():
    """The tests' plain plan on a case worked by hand: page size 4, request 0 shrinks
    from 9 to 3 (pages 7, 2 go back), 1 grows from 4 to 6 (takes 2), 2 from 0 to 9
    (takes 7, 5, 1)."""
    r = ref.plan([9, 4, 0], [3, 6, 9], [[4, 7, 2], [0, -1, -1], [-1, -1, -1]],
                 [1, 5, -1, -1, -1, -1, -1, -1], 2, 4, 12)
    assert r["table"] == [[4, 7, 2], [0, 2, -1], [7, 5, 1]]
    assert r["slot_map"] == [8, 9, 28, 29, 30, 31, 20, 21, 22, 23, 4, -1]
    assert r["positions"] == [4, 5, 0, 1, 2, 3, 4, 5, 6, 7, 8, 0]
    assert r["new_count"] == [0] and r["info"] == [11, 4, 2, 0] and r["cu_new"] == [0, 0, 2, 11]
