"""CPU: further refusals of the paged-cache entry points, by the C ABI (the pointers
are never followed) and by the Python binding."""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn
from gated_delta_rule_106_b200 import _build

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def test_plan_capacity_is_refused_before_outputs_are_made(lib):
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_page_plan(i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16,
                          token_capacity=(1 << 30) + 1)
    assert e.value.status == INVALID


def test_a_given_stream_does_not_change_refusals():
    """With a stream the same exceptions as without: missing tensors, wrong types,
    tensors on the CPU."""
    q = torch.zeros(5, 8, 64).half()
    c = torch.zeros(3, 16, 2, 64).half()
    for kw in ({}, dict(stream=0)):
        with pytest.raises(ValueError, match="give q"):
            gdn.gdn_qk_norm_rope(None, None, None, **kw)
        with pytest.raises(TypeError, match="q: a torch.Tensor is needed"):
            gdn.gdn_qk_norm_rope([1.0], None, None, **kw)
        with pytest.raises(TypeError, match="lens: a torch.Tensor is needed"):
            gdn.gdn_page_plan([3], i32(1), i32(1, 4), i32(9), i32(1), 16, token_capacity=8, **kw)
        with pytest.raises(TypeError, match="q: a torch.Tensor is needed"):
            gdn.gdn_paged_attention_decode(None, c, c, i32(5, 2), i32(5), **kw)
        for call in (lambda: gdn.gdn_qk_norm_rope(q, None, None, **kw),
                     lambda: gdn.gdn_page_plan(i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16,
                                               token_capacity=8, **kw),
                     lambda: gdn.gdn_paged_attention_decode(q, c, c, i32(5, 2), i32(5), **kw)):
            with pytest.raises(ValueError, match="CUDA tensors only"):
                call()


def test_rope_frequencies_of_infinite_arguments_are_refused(lib):
    """An infinite base or bound would give NaN frequencies."""
    inf = float("inf")
    call = lambda R=64, base=1e7, f=1.0, ctx=8192.0, hi=32.0, lo=1.0: (  # noqa: E731
        lib.gdn_rope_inv_freq(R, base, f, ctx, hi, lo, None, None))
    for kw in (dict(base=inf), dict(f=inf), dict(ctx=inf), dict(hi=inf), dict(lo=-inf),
               dict(hi=inf, lo=-inf), dict(base=float("nan"))):
        assert call(**kw) == INVALID, kw
        # the same without a table to make
        assert call(R=0, **kw) == INVALID, kw
    assert call(R=0) == OK
    assert call(R=0, ctx=0.0, hi=inf) == OK                  # the bounds are not used


A = 1 << 40                        # an aligned address that nothing follows
STEP = 1 << 34


def test_outputs_over_other_arguments_are_refused(lib):
    """The decode writes o and lse while it reads lengths, tables, queries and gates, and
    its workspace throughout; the append writes q_out while it reads everything else.
    Returned before any launch: were one of them taken, the addresses would be followed."""
    need = lib.gdn_paged_attention_decode_workspace(24, 4, 256)
    base = dict(q=A, qs=24 * 256, kc=A + STEP, kp=65536, kt=1024, kh=256, vc=A + 2 * STEP, vp=65536,
                vt=1024, vh=256, kd=2, P=64, page=64, table=A + 3 * STEP, row=16, width=16,
                lens=A + 4 * STEP, gate=A + 5 * STEP, gs=24 * 256, N=4, Hq=24, Hkv=4, D=256,
                scale=0.0625, o=A + 6 * STEP, od=0, lse=A + 7 * STEP, ws=A + 8 * STEP, wb=need,
                s=None)
    o, lse, ws, row = base["o"], base["lse"], base["ws"], 24 * 256 * 2
    for kw in (dict(table=o), dict(table=o + 4 * row - 4), dict(lens=o), dict(lse=o + 64),
               dict(ws=o), dict(ws=o + 4 * row - 16), dict(ws=o - (need - 16) // 16 * 16),
               dict(q=lse), dict(gate=lse), dict(table=lse), dict(lens=lse), dict(ws=lse),
               dict(q=ws), dict(gate=ws), dict(table=ws + 16), dict(lens=ws + need // 16 * 16 - 16)):
        assert lib.gdn_paged_attention_decode(*{**base, **kw}.values()) == INVALID, kw
    base = dict(q=A, qs=24 * 256, k=A + STEP, ks=1024, v=A + 2 * STEP, vs=1024, xd=0, wq=A + 6 * STEP,
                wk=A + 7 * STEP, wd=1, eps=1e-6, pos=A + 8 * STEP, axes=3, inv=A + 9 * STEP, R=64,
                inter=0, rs=1.0, slots=A + 10 * STEP, T=8, Hq=24, Hkv=4, D=256, qo=A + 3 * STEP,
                kc=A + 4 * STEP, kp=16384, kt=1024, kh=256, vc=A + 5 * STEP, vp=16384, vt=1024,
                vh=256, P=8, page=16, od=2, s=None)
    for name in ("wq", "wk", "pos", "inv", "slots"):
        for at in (base["qo"], base["qo"] + 8 * row - 16):
            assert lib.gdn_qk_norm_rope(*{**base, name: at}.values()) == INVALID, name
