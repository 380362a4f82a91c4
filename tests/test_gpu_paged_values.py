"""GPU: infinite and NaN values in the paged-cache operators: which outputs they reach."""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn
import _paged as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
f64 = ref.f64


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [2, 20, 34, 64, 126])
def test_turned_dims_leave_the_others_alone(R, interleaved, value):
    """Without a norm, dims behind rope_dims pass unchanged (rounded to bf16, exactly here)
    whatever a dim beside them holds, and a turned pair depends on itself alone."""
    T, H, D = 3, 2, 128
    x = torch.randn(T, H, D, device=DEV).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 5
    inv = gdn.gdn_rope_inv_freq(R, 1e4)
    kw = dict(positions=pos, inv_freq=inv, interleaved=interleaved, out_dtype=BF16)
    clean = gdn.gdn_qk_norm_rope(x, None, None, **kw)
    assert torch.equal(clean[..., R:], x[..., R:])
    for d in range(D):
        y = x.clone()
        y[1, 1, d] = value
        got = gdn.gdn_qk_norm_rope(y, None, None, **kw)
        reached = {d}
        if d < R:
            half = R // 2
            reached.add(d ^ 1 if interleaved else (d + half) % R)
        others = [i for i in range(D) if i not in reached]
        assert torch.equal(got[1, 1, others], clean[1, 1, others]), d
        assert torch.equal(got[[0, 2]], clean[[0, 2]]) and torch.equal(got[1, 0], clean[1, 0])
        if d >= R:
            assert torch.equal(got[1, 1, d].nan_to_num(7.0, 8.0, 9.0),
                               y[1, 1, d].nan_to_num(7.0, 8.0, 9.0))
        else:
            assert not bool(got[1, 1, sorted(reached)].isfinite().any())
