"""The device that last_device_error and selftest_wait_limit take: none, an
index, a string or a torch.device, as torch.cuda.current_stream takes them."""
import pytest
import torch

import exact_tiled_attention_24_gb300 as fa
from test_binding_checks import FakeLib

FORMS = [(None, 1), (0, 0), (3, 3), ("cuda", 1), ("cuda:2", 2), (torch.device("cuda"), 1), (torch.device("cuda", 2), 2)]


@pytest.mark.parametrize("device,index", FORMS, ids=[str(f[0]) for f in FORMS])
def test_every_form_of_a_device(monkeypatch, device, index):
    asked, lib = [], FakeLib()
    monkeypatch.setattr(fa, "lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: asked.append(i) or 0, raising=False)
    assert fa.last_device_error(device) == 0
    fa.selftest_wait_limit(device)
    assert asked == [index, index] and lib.calls == ["fa_last_device_error", "fa_selftest_wait_limit"]


@pytest.mark.gpu
def test_on_the_gpu():
    x = torch.ones((2, 8), device="cuda")
    fa.softmax_online(x)
    for device in (None, 0, "cuda", "cuda:0", x.device):
        assert fa.last_device_error(device) == 0
