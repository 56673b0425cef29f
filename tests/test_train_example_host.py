"""What expert_ffn of the training example refuses: answered before anything runs, without a GPU."""
import pytest
import torch

from examples.train_experts import expert_ffn

T, H, INTER, E, TOPK = 5, 64, 32, 3, 2


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on a CUDA device."""

    @property
    def is_cuda(self):
        return True


def good():
    return {"x": torch.zeros(T, H, dtype=torch.bfloat16), "route_weights": torch.zeros(T, TOPK),
            "w_gateup": torch.zeros(E, 2 * INTER, H, dtype=torch.bfloat16),
            "w_down": torch.zeros(E, H, INTER, dtype=torch.bfloat16),
            "expert_ids": torch.zeros(T, TOPK, dtype=torch.int32)}


def on_device(args):
    return {name: t.as_subclass(OnDevice) for name, t in args.items()}


def test_good_operands_pass_the_checks(monkeypatch):
    from examples import train_experts
    monkeypatch.setattr(train_experts._ExpertFFN, "apply", lambda *args: args)
    assert len(expert_ffn(**on_device(good()))) == 5


@pytest.mark.parametrize("name,dtype", [("x", torch.float16), ("x", torch.float32), ("route_weights", torch.bfloat16),
                                        ("route_weights", torch.float64), ("expert_ids", torch.int64),
                                        ("w_gateup", torch.float16), ("w_down", torch.float32)])
def test_types(name, dtype):
    args = good()
    args[name] = args[name].to(dtype)
    with pytest.raises(ValueError, match=f"{name} is torch"):
        expert_ffn(**on_device(args))


@pytest.mark.parametrize("name", ["x", "route_weights", "expert_ids", "w_gateup", "w_down"])
def test_shapes_and_devices(name):
    for cut in (lambda t: t[:-1], lambda t: t[:, :-1], lambda t: t[0]):
        args = good()
        args[name] = cut(args[name])
        with pytest.raises(ValueError, match="expected|takes"):
            expert_ffn(**on_device(args))
    args = on_device(good())
    args[name] = good()[name]
    with pytest.raises(ValueError, match=f"{name} is on cpu"):
        expert_ffn(**args)


def test_widths_that_no_group_divides():
    args = good()
    args["x"], args["w_gateup"], args["w_down"] = args["x"][:, :40], args["w_gateup"][:, :, :40], args["w_down"][:, :40]
    with pytest.raises(ValueError, match="multiples of 32"):
        expert_ffn(**on_device(args))
