"""What a call of the losses or of the optimizer with ``stream=`` allocates
belongs to that stream, on the CPU with a fake library and fake streams."""

import pytest
import torch

from fp8_communication_compression_gb300 import AdamW, api
from test_stream_memory import CURRENT, SIDE, Noted, Side, notes, t  # noqa: F401 (a fixture)


class Placed(Noted):
    def get_device(self):
        return 0


def p(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Placed)


x, a, f = lambda: t((4, 256)), lambda: t(4, torch.int64), lambda: t(4, torch.float32)
CALLS = {
    "token_logprob": lambda s: api.token_logprob(x(), a(), stream=s),
    "token_logprob_backward": lambda s: api.token_logprob_backward(f(), x(), a(), f(), stream=s),
    "policy_loss": lambda s: api.policy_loss(x(), a(), f(), f(), f(), stream=s),
    "preference_loss": lambda s: api.preference_loss(x(), a(), t(3, torch.int64), stream=s),
    "grad_norm": lambda s: api.grad_norm([p(4)], stream=s),
    "AdamW.step": lambda s: STEP(s),
}


def STEP(s):
    opt = AdamW([p(4)], max_norm=1.0)
    return opt.step([p(4)], stream=s)


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_side_stream(notes, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(api, "_norm_partials_bytes", lambda n: 512)
    side = Side()
    CALLS[name](side)
    made = [m for m in notes["made"]]
    assert made and all(m.made_on is side for m in made), name
