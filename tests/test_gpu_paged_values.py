"""GPU: infinite and NaN values in the paged-cache operators: which outputs they reach."""
import math

import pytest
import torch

import gated_delta_rule_106_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


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


def paged(k_rows, v_rows, page):
    """Caches, table and lengths of sequences with the given rows [N, L, H_kv, D]."""
    N, L, H, D = k_rows.shape
    held = -(-L // page)
    caches = []
    for rows in (k_rows, v_rows):
        c = torch.full((N * held, page, H, D), float("nan"), dtype=rows.dtype, device=DEV)
        c.view(N, held * page, H, D)[:, :L] = rows
        caches.append(c)
    table = torch.arange(N * held, dtype=torch.int32, device=DEV).view(N, held)
    return *caches, table, torch.full((N,), L, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 4, 4), (64, 16, 1), (128, 6, 2), (128, 16, 1),
                                        (256, 24, 4), (256, 16, 1)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weights_keep_their_bits_in_fp32_outputs(D, H_q, H_kv, dtype):
    """Weights go into the product with V in 16-bit parts, two for fp16 and three for
    bf16; for fp32 outputs each part counts. Two tokens, the first with score 0 and value
    0, the second with score -j / 64 for integers j, exact in fp32, so that an output is
    w / (1 + w) v with w = 2^x, x = -j / 64 log2 e, and its error is that of
      the weights' arguments: x (the scale's and the product's rounding, 2^-24 |x| each)
        and x + 11 (2^-21), times ln 2; the exponentials 2^-22 each;
      the parts: 2^-22 for two of fp16 (each leaves 2^-11), less for three of bf16;
      their products' sums, the warps' sums, the quotient and its product: 8 of 2^-23.
    Two parts of bf16 leave up to 2^-18, one part of fp16 2^-11: emulated below, both are
    past twice that bound."""
    N = 256 // H_q
    j = (torch.arange(N * H_q, device=DEV) * 37 % 256 + 1).view(N, H_q)
    q = torch.zeros(N, H_q, D, device=DEV, dtype=dtype)
    q[..., 3] = j.to(dtype)
    k = torch.zeros(N, 2, H_kv, D, device=DEV, dtype=dtype)
    k[:, 1, :, 3] = -1
    v = torch.zeros_like(k)
    v[:, 1] = (1 + torch.rand(N, H_kv, D, device=DEV)).to(dtype)
    assert torch.equal(q[..., 3].long(), j)
    o = gdn.gdn_paged_attention_decode(q, *paged(k, v, 16), scale=1 / 64, o_dtype=F32)
    w = torch.exp(-j.double() / 64)[..., None]
    want = w / (1 + w) * v[:, 1].double().repeat_interleave(H_q // H_kv, dim=1)
    x = j.double()[..., None] / 64 / math.log(2)
    bound = math.log(2) * (2 * 2.0 ** -24 * x + 2.0 ** -21) + 2 * 2.0 ** -22 + 8 * 2.0 ** -23
    bound = bound + (2.0 ** -22 if dtype == F16 else 0.0)
    off = (o.double() - want).abs() / want
    assert bool((off <= bound).all()), float((off / bound).max())
    # the same with a part left out
    p = torch.exp2(11 - x)
    left = p.clone()
    for _ in range(1 if dtype == F16 else 2):
        left = left - left.to(dtype).double()
    assert float(((left / p).abs() / bound).max()) > 2


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_and_large_cached_values(dtype):
    """An infinite value of a row among a sequence's makes its dim infinite or NaN in the
    heads that share it (a weight enters in parts, high * inf + low * inf: NaN where the
    low part is not above 0) and nothing else; values up to 2^112 / length of bf16 caches
    are no different from others."""
    g = torch.Generator(device=DEV).manual_seed(5)
    N, L, H_q, H_kv, D = 3, 70, 4, 2, 64
    q, k, v = (torch.randn(*n, D, device=DEV, generator=g).to(dtype)
               for n in ((N, H_q), (N, L, H_kv), (N, L, H_kv)))
    args = paged(k, v, 16)
    clean = gdn.gdn_paged_attention_decode(q, *args, o_dtype=F32)
    assert bool(clean.isfinite().all())
    for at in (0, 33, L - 1):
        w = v.clone()
        w[1, at, 1, 7] = float("inf")
        o = gdn.gdn_paged_attention_decode(q, *paged(k, w, 16), o_dtype=F32)
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[1, 2:, 7] = True
        assert not bool(o[hit].isfinite().any()) and torch.equal(o[~hit], clean[~hit])
    if dtype == BF16:
        big = 2.0 ** 100
        o = gdn.gdn_paged_attention_decode(q, *paged(k, v * big, 16), o_dtype=F32)
        assert torch.equal(o, clean * big)
