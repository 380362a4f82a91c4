"""GPU: what the binding of the paged-cache calls does with tensors and arguments
that the library cannot take. Nothing is launched in these calls."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

import gated_delta_rule_106_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def state():
    """Arguments of the three calls, by name."""
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    h = lambda *n: torch.zeros(*n, dtype=torch.float16, device=DEV)  # noqa: E731
    return dict(lens=i(3), want=i(3), table=i(3, 4), free=i(9), count=i(1), q=h(3, 4, 64),
                k=h(3, 2, 64), v=h(3, 2, 64), kc=h(9, 16, 2, 64), vc=h(9, 16, 2, 64), slots=i(3),
                w=torch.ones(64, device=DEV), pos=i(3),
                inv=torch.ones(16, dtype=torch.float64, device=DEV),
                gate=torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV),
                lse=torch.zeros(3, 4, device=DEV), o=h(3, 4, 64),
                ws=torch.zeros(gdn.gdn_paged_attention_decode_workspace(4, 2, 64),
                               dtype=torch.uint8, device=DEV))


def plan(s):
    gdn.gdn_page_plan(s["lens"], s["want"], s["table"], s["free"], s["count"], 16,
                      token_capacity=8)


def rope(s):
    gdn.gdn_qk_norm_rope(s["q"], s["k"], s["v"], s["kc"], s["vc"], slot_map=s["slots"],
                         q_norm_w=s["w"], k_norm_w=s["w"], positions=s["pos"], inv_freq=s["inv"])


def decode(s):
    gdn.gdn_paged_attention_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                   gate=s["gate"], o=s["o"], lse=s["lse"], workspace=s["ws"])


@pytest.mark.parametrize("call,names", [
    (plan, "lens want table free count"), (rope, "q k v kc vc slots w pos inv"),
    (decode, "q kc vc table lens gate lse o ws")])
def test_tensors_without_an_address(call, names):
    """Tensors that stand for others (of a mode without memory, or of a batch that is
    mapped over): an exception, whichever argument it is."""
    for name in names.split():
        s = state()
        with FakeTensorMode() as mode:
            fake = mode.from_tensor(s[name])
        with pytest.raises((ValueError, RuntimeError), match="memory|data pointer|storage"):
            call(dict(s, **{name: fake}))
        with pytest.raises((ValueError, RuntimeError), match="memory|data pointer|storage"):
            torch.vmap(lambda t: call(dict(s, **{name: t})))(s[name].unsqueeze(0))
    call(state())
    torch.cuda.synchronize()


def test_exceptions_keep_their_types():
    """Running out of memory for an output, and what a mode raises while one is made."""
    s = state()
    try:
        torch.cuda.set_per_process_memory_fraction(0.005)
        with pytest.raises(torch.OutOfMemoryError):
            gdn.gdn_page_plan(s["lens"], s["want"], s["table"], s["free"], s["count"], 16,
                              token_capacity=1 << 30)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)

    class Stop(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            raise KeyError("stop")

    for call in (plan, rope, decode):
        t = dict(s, o=None)
        with Stop(), pytest.raises(KeyError, match="stop"):
            call(t)
    plan(s)
    torch.cuda.synchronize()
