"""GPU: a bounded wait inside the paged decode that runs out is reported to the
caller, leaves NaN in every row with tokens and nothing outside the outputs, and
leaves the workspace and the context usable.

The copying and computing warps of a CTA wait for one another on mbarriers, each
wait bounded by gdn_set_wait_limit_ns. The test lowers that bound to 1 ns, less
than any read of global memory takes, so waits run out: no fault, no hang, just
the designed way out. The workspace holds set bits beforehand: entries that
this call did not write must not be followed.
"""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("D,H_q,H_kv,page,dtype,N,hi", [
    (256, 24, 4, 64, torch.float16, 6, 900),        # copied by TMA
    (128, 8, 4, 7, torch.bfloat16, 5, 700),         # by cp.async
    (64, 16, 16, 48, torch.float16, 61, 2900),      # CTAs without work, to be cancelled
    (256, 8, 4, 16, torch.float16, 40, 4300),
    (256, 8, 4, 16, torch.float16, 64, 4300),       # ranges that other CTAs take over
    (128, 16, 8, 9, torch.bfloat16, 64, 4300)])     # the same by cp.async
def test_waits_that_run_out(D, H_q, H_kv, page, dtype, N, hi):
    g = torch.Generator(device=DEV).manual_seed(D + page)
    width = -(-hi // page)
    P = width + 3
    kc, vc = (torch.randn(P, page, H_kv, D, device=DEV, generator=g).to(dtype) for _ in range(2))
    table = torch.stack([torch.randperm(P, device=DEV, generator=g)[:width]
                         for _ in range(N)]).to(torch.int32)
    lens = torch.randint(hi // 2, hi + 1, (N,), device=DEV, generator=g, dtype=torch.int32)
    lens[1], lens[2] = 0, width * page + 1          # empty; out of range
    q = torch.randn(N, H_q, D, device=DEV, generator=g).to(dtype)
    gate = torch.randn(N, H_q, D, device=DEV, generator=g).bfloat16()
    need = gdn.gdn_paged_attention_decode_workspace(H_q, H_kv, D)

    def run(ws):
        o = torch.full((N + 2, H_q, D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((N + 2, H_q), 7.0, device=DEV)
        gdn.gdn_paged_attention_decode(q, kc, vc, table, lens, gate=gate, o=o[1:-1],
                                       lse=lse[1:-1], workspace=ws[:need])
        st = gdn.gdn_attention_status(ws)
        assert bool((ws[need:] == 255).all())
        for t in (o, lse):
            assert bool((t[[0, -1]] == 7.0).all())
        return o[1:-1], lse[1:-1], st

    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    o_ref, lse_ref, st = run(ws)
    assert st == -1                                  # the length out of range
    with_tokens = torch.ones(N, dtype=torch.bool, device=DEV)
    with_tokens[1] = False
    assert bool(o_ref[2].isnan().all()) and bool(o_ref[3:].isfinite().all())
    try:
        gdn.gdn_set_wait_limit_ns(1)
        for fill in (255, 1, None):                  # None: what the last call left
            if fill is not None:
                ws[:need] = fill
            o, lse, st = run(ws)
            assert st == gdn.GDN_ERR_TIMEOUT, gdn.gdn_status_string(st)
            assert bool(o[with_tokens].isnan().all()) and bool(lse[with_tokens].isnan().all())
            assert not bool(o[1].any()) and bool((lse[1] == float("-inf")).all())
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    def same(o, lse):
        return (torch.equal(o.nan_to_num(9.0), o_ref.nan_to_num(9.0)) and
                torch.equal(lse.nan_to_num(9.0, neginf=8.0), lse_ref.nan_to_num(9.0, neginf=8.0)))

    o, lse, st = run(ws)
    assert st == -1 and same(o, lse)
    # bounds that some waits keep and others do not: all or nothing
    try:
        for ns in (300, 1000, 2000, 4000, 8000, 16000, 64000, 500000):
            gdn.gdn_set_wait_limit_ns(ns)
            for fill in (255, 0, None):
                if fill is not None:
                    ws[:need] = fill
                o, lse, st = run(ws)
                if st == gdn.GDN_ERR_TIMEOUT:
                    assert bool(o[with_tokens].isnan().all() and lse[with_tokens].isnan().all())
                    assert not bool(o[1].any()) and bool((lse[1] == float("-inf")).all())
                else:
                    assert st == -1 and same(o, lse), ns
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    o, lse, st = run(ws)
    assert st == -1 and same(o, lse)
