"""GPU: the paged decode right behind the call that makes its lengths, again and again
on the same buffers, with no synchronisation between: rows without tokens are written
by a kernel that comes in early and has to see the lengths of its own step."""
import pytest
import torch

import gated_delta_rule_106_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("D,H_q,H_kv,page,N", [(64, 2, 1, 16, 700), (256, 24, 4, 16, 40)])
@pytest.mark.parametrize("by_plan", [True, False])
def test_lengths_written_by_the_call_before(D, H_q, H_kv, page, N, by_plan):
    g = torch.Generator(device=DEV).manual_seed(N)
    width, P = 4, 64
    dt = torch.float16
    kc, vc = (torch.randn(P, page, H_kv, D, device=DEV, generator=g).to(dt) for _ in range(2))
    table = torch.randint(P, (N, width), device=DEV, generator=g, dtype=torch.int32)
    q = torch.randn(N, H_q, D, device=DEV, generator=g).to(dt)
    gate = torch.randn(N, H_q, D, device=DEV, generator=g).bfloat16()
    ws = torch.empty(gdn.gdn_paged_attention_decode_workspace(H_q, H_kv, D), dtype=torch.uint8,
                     device=DEV)
    lens = torch.empty(N, dtype=torch.int32, device=DEV)
    # a third of the rows empty, others in each step
    steps = [torch.randint(1, width * page + 1, (N,), device=DEV, generator=g, dtype=torch.int32)
             for _ in range(5)]
    for i, s in enumerate(steps):
        s[torch.rand(N, device=DEV, generator=g) < 0.33] = 0
        s[i] = 0
    zero = torch.zeros(N, dtype=torch.int32, device=DEV)
    spare = torch.arange(N * width, dtype=torch.int32, device=DEV)
    full = torch.tensor([N * width], dtype=torch.int32, device=DEV)
    room = N * width * page
    out = dict(cu_new=torch.empty(N + 1, dtype=torch.int32, device=DEV),
               slot_map=torch.empty(room, dtype=torch.int32, device=DEV),
               new_count=torch.empty(1, dtype=torch.int32, device=DEV))
    scratch = torch.empty(N, width, dtype=torch.int32, device=DEV)

    def step(i, o):
        if by_plan:
            gdn.gdn_page_plan(zero, steps[i], scratch, spare, full, page, new_lens=lens, **out)
        else:
            lens.copy_(steps[i])
        gdn.gdn_paged_attention_decode(q, kc, vc, table, lens, gate=gate, o=o, workspace=ws)

    want = []
    for i in range(5):
        o = torch.empty(N, H_q, D, dtype=torch.bfloat16, device=DEV)
        step(i, o)
        torch.cuda.synchronize()
        assert torch.equal(lens, steps[i])
        assert torch.equal((o == 0).all(-1).all(-1), steps[i] == 0)
        want.append(o)
    got = [torch.full_like(want[0], 7.0) for _ in range(200)]
    order = torch.randint(5, (200,), generator=torch.Generator().manual_seed(1)).tolist()
    for o, i in zip(got, order):
        step(i, o)
    torch.cuda.synchronize()
    for n, (o, i) in enumerate(zip(got, order)):
        assert torch.equal(o, want[i]), n
