"""What the optimiser hands to the library, without a GPU."""

import inspect

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from block_sparse_attention_sparge_gb300 import train as T


@pytest.fixture
def calls(monkeypatch):
    """The calls of sparge_muon_step, checked against its signature."""
    seen, signature = [], inspect.signature(B.sparge_muon_step)

    def step(*args, **kw):
        bound = signature.bind(*args, **kw)
        bound.apply_defaults()
        seen.append(bound.arguments)

    monkeypatch.setattr(B, "sparge_muon_step", step)
    return seen


def _weights():
    ws = [torch.nn.Parameter(torch.randn(4, 6)) for _ in range(2)]
    for w in ws:
        w.grad = torch.randn(4, 6)
    return ws


def test_under_a_schedule(calls):
    opt = T.Muon(_weights(), lr=0.1, momentum=0.8, weight_decay=0.2)
    schedule = torch.optim.lr_scheduler.StepLR(opt, 1, gamma=0.5)
    for lr in (0.1, 0.05, 0.025):
        opt.step()
        schedule.step()
        assert calls[-1]["lr"] == pytest.approx(lr)
        assert calls[-1]["momentum"] == 0.8 and calls[-1]["weight_decay"] == 0.2
    # a checkpoint brings the schedule's key along
    other = T.Muon(_weights(), lr=0.7)
    other.load_state_dict(opt.state_dict())
    other.step()
    assert calls[-1]["lr"] == pytest.approx(0.0125)


def test_named_parameters_and_keys_of_the_users_own(calls):
    module = torch.nn.Linear(6, 4, bias=False)
    module.weight.grad = torch.randn(4, 6)
    opt = T.Muon([dict(params=list(module.parameters()), lr=0.3, label="attention")])
    opt.step()
    assert calls[-1]["lr"] == 0.3
    try:
        opt = T.Muon(module.named_parameters())
    except TypeError:
        pytest.skip("this torch takes no named parameters")
    opt.step()
    assert len(calls) == 2 and calls[-1]["weights"][0] is module.weight


def test_which_side_of_a_weight_its_inputs_are(calls):
    a, b = _weights()
    opt = T.Muon([dict(params=[a]), dict(params=[b], inputs_first=True)])
    opt.step()
    assert [c["inputs_first"] for c in calls] == [False, True]
    state = opt.state_dict()
    for group in state["param_groups"]:
        del group["inputs_first"]
    opt.load_state_dict(state)
    opt.step()
    assert [c["inputs_first"] for c in calls[2:]] == [False, False]
