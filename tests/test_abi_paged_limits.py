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
