"""The mixture-of-experts layer's binding on the CPU: what it asks the library for, with the call itself left out."""
import pytest
import torch

import structured_sparse_gemm_amd as hinm

BF16 = torch.bfloat16


@pytest.fixture
def asked(monkeypatch):
    """Sizes of the workspaces that moe_layer asks for; its calls return at once."""
    sizes = []
    monkeypatch.setattr(hinm, "_on_gpu", lambda dev: None)
    monkeypatch.setattr(hinm, "_stream_ptr", lambda dev: 0)
    monkeypatch.setattr(hinm, "_call", lambda dev, fn, *args: None)
    monkeypatch.setattr(hinm, "_sized_workspace", lambda dev, stream, need: sizes.append(need))
    return sizes


def _stack(cout, cin, n=4):
    p = hinm.plan(cout, cin, 64, 0.75, 0.55)
    return hinm.Experts.stack([hinm.alloc_packed(p, "cpu") for _ in range(n)])


def test_workspace_is_of_the_call_at_hand(asked):
    """A gate's sizes are not those that an earlier call with other projections asked for."""
    gate, up, down = _stack(1024, 128), _stack(1024, 128), _stack(128, 1024)
    x, logits = torch.zeros(128, 3, dtype=BF16), torch.zeros(4, 3)
    hinm.moe_layer(x, logits, gate, _stack(192, 128), _stack(128, 192), 2)    # refused by the library: unequal shapes
    hinm.moe_layer(x, logits, gate, up, down, 2)
    hinm.moe_layer(x, logits, gate, up, down, 2)
    small = hinm.moe_layer_workspace_bytes(hinm.plan(192, 128, 64, 0.75, 0.55), hinm.plan(128, 192, 64, 0.75, 0.55), 4, 3, 2)
    need = hinm.moe_layer_workspace_bytes(up.plan, down.plan, 4, 3, 2)
    assert asked == [small, need, need] and small < need


class _Tagged(hinm.Experts):
    """A user's own stack."""


def test_a_subclass_is_a_stack_of_its_kind(asked):
    """Stacks are told apart by their class, not by its name."""
    gate, up, down = _stack(192, 128), _stack(192, 128), _stack(128, 192)
    tagged = _Tagged(gate.plan, **{k: getattr(gate, k) for k in hinm._packed_shapes(gate.plan)})
    x, logits = torch.zeros(128, 3, dtype=BF16), torch.zeros(4, 3)
    hinm.moe_layer(x, logits, tagged, up, down, 2)
    assert len(asked) == 1

    class Experts:
        n_experts = 4
    with pytest.raises(ValueError, match="of one kind"):
        hinm.moe_layer(x, logits, Experts(), Experts(), Experts(), 2)
