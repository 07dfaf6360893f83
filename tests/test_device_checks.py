"""The binding's check that a call's tensors lie on one CUDA device, on stand-ins: no GPU is reached."""

import inspect
import re

import pytest

import paged_kv_gqa_attn_gb300 as pa


class _On:
    """A tensor as the check sees it."""

    def __init__(self, index):
        self.device = f"cuda:{index}" if index >= 0 else "cpu"
        self.index = index

    def get_device(self):
        return self.index


def test_tensors_on_two_devices_are_named():
    with pytest.raises(ValueError, match=r"one CUDA device.*'q': 'cuda:0'.*'out': 'cuda:1'"):
        pa._one_device(None, _On(0), None, _On(1), names="q k_scale out")
    with pytest.raises(ValueError, match=r"'b': 'cpu'"):
        pa._one_device(None, a=_On(0), b=_On(-1))


def test_a_host_tensor_is_refused_wherever_it_stands():
    for order in ((-1, 0), (0, -1), (-1, -1), (-1,)):
        with pytest.raises(ValueError, match="one CUDA device"):
            pa._one_device(None, *[_On(i) for i in order], names="a b")
    with pytest.raises(ValueError, match="got none"):
        pa._one_device(None, None, names="a")


def test_every_call_names_each_tensor_that_it_passes():
    text = re.sub(r"\s+", " ", inspect.getsource(pa))
    calls = re.findall(r"with _one_device\(stream, ([^=]*?), names=\"([^\"]*)\"\)", text)
    assert len(calls) == 5
    for args, names in calls:
        assert args.replace("*outs", "k_out, v_out").split(", ") == names.split()
