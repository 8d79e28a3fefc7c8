"""Operands and workspaces of the training-step calls that lie elsewhere are
refused before anything reaches the library, which is replaced by a recorder
here, so that no pointer gets to a kernel even where a check is missing."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, D, E = 8, 64, 16
ROLES = {
    "moe_layer_norm": dict(x=(T, D), weight=(D,), bias=(D,), residual=(T, D), out=(T, D), stats=(2, T), z=(T, D)),
    "moe_layer_norm_backward": dict(dy=(T, D), z=(T, D), stats=(2, T), weight=(D,), dz=(T, D), workspace=(1 << 16,)),
    "moe_router_loss": dict(logits=(T, E), counts=(E,), mask=(T,), out=(T, E), losses=(2,), workspace=(1 << 17,)),
    "moe_grad_norm": dict(tensors=(1,), out=(2,), workspace=(1 << 16,)),
    "moe_adamw_step": dict(plan=(1,), clip=(2,), hyper=(8,)),
}
DTYPES = dict(workspace=torch.uint8, counts=torch.int32, mask=torch.bool)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


class Elsewhere(torch.Tensor):
    """A CUDA tensor that says it is on the next device."""

    def get_device(self):
        return 1


@pytest.fixture
def moe(monkeypatch):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_expert_gb300 as m
    monkeypatch.setattr(m._lib, "lib", Recorder())
    return m


def arguments(moe, name):
    args = {role: torch.zeros(shape, dtype=DTYPES.get(role, torch.float32), device="cuda")
            for role, shape in ROLES[name].items()}
    if name == "moe_grad_norm":
        args["tensors"] = moe.moe_tensor_list([args["tensors"]])
    if name == "moe_adamw_step":
        p = args["plan"]
        args["plan"] = moe.moe_adamw_plan([p], [p.clone()], **moe.moe_adamw_state([p]))
    return args


@pytest.mark.parametrize("name,role", [(n, r) for n in ROLES for r in ROLES[n] if r not in ("tensors", "plan")])
def test_operands_elsewhere(moe, name, role):
    args, calls = arguments(moe, name), moe._lib.lib.calls
    getattr(moe, name)(**args)
    assert calls == [name]
    for other in (args[role].cpu(), args[role].as_subclass(Elsewhere)):
        with pytest.raises(ValueError):
            getattr(moe, name)(**{**args, role: other})
    assert calls == [name]


@pytest.mark.parametrize("name", [n for n in ROLES if "workspace" in ROLES[n]])
def test_workspaces_with_gaps(moe, name):
    args = arguments(moe, name)
    args["workspace"] = torch.zeros(2 << 17, dtype=torch.uint8, device="cuda")[::2]
    with pytest.raises(ValueError):
        getattr(moe, name)(**args)
    assert not moe._lib.lib.calls


@pytest.mark.parametrize("name", list(ROLES))
def test_another_current_device(moe, name, monkeypatch):
    args = arguments(moe, name)
    monkeypatch.setattr(moe._lib, "_current_device", lambda: 1)
    with pytest.raises(ValueError):
        getattr(moe, name)(**args)
    with pytest.raises(ValueError):
        getattr(moe, name)(**args, stream=torch.cuda.Stream())
    assert not moe._lib.lib.calls
