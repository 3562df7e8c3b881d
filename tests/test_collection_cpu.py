"""Which tests run where: the ones that need a device only where there is one,
the ones that must not meet a device only where there is none."""
import pathlib

import conftest
import pytest
import torch


class _Item:
    def __init__(self, path, name, gpu=False):
        self.path, self.originalname = pathlib.Path("/somewhere/tests") / path, name
        self.keywords = {"gpu": True} if gpu else {}
        self.markers = []

    def add_marker(self, m):
        self.markers.append(m)


@pytest.mark.parametrize("device", [False, True])
def test_skips(monkeypatch, device):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: device)
    unsafe = [_Item("test_head_cpu.py", n) for n in ("test_sizes", "test_pointers", "test_without_a_device")]
    plain = [_Item("test_head_cpu.py", "test_workspace_sizes"), _Item("test_abi_cpu.py", "test_sizes")]
    gpu = [_Item("test_head_gpu.py", "test_loss", gpu=True)]
    conftest.pytest_collection_modifyitems(None, unsafe + plain + gpu)
    skipped = [bool(i.markers) for i in unsafe + plain + gpu]
    assert skipped == ([True] * 3 + [False] * 3 if device else [False] * 5 + [True])
    for i in unsafe + gpu:
        for m in i.markers:
            assert m.name == "skip" and m.kwargs["reason"]
