"""What the binding of the norms, dropout and the balance loss does before a call (CPU only)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lp():
    import lm_head_linear_tcgen05_gb300 as mod
    return mod


def test_the_current_device_is_asked_for_by_its_public_name(lp, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    assert lp._on(torch.device("cuda:3")) is lp._SAME_DEVICE
    assert isinstance(lp._on(torch.device("cuda:1")), torch.cuda.device)
