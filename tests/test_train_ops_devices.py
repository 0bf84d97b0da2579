"""The operators' binding refuses tensors of another device than the current one (host: stand-ins for tensors)."""
import pytest
import torch

import fully_sharded_gb300 as fs

BF16, F32 = torch.bfloat16, torch.float32


class On:
    """A CPU tensor that says it lies on a CUDA device."""

    is_cuda = True

    def __init__(self, index, *shape, dtype=BF16):
        self._t, self._index = torch.zeros(*shape, dtype=dtype), index

    def get_device(self):
        return self._index

    @property
    def device(self):
        return torch.device("cuda", self._index)

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture(autouse=True)
def first_device(monkeypatch):
    """Device 0 is the current one; a call that is not refused does not reach the library."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def reached(*args):
        raise AssertionError("a tensor of another device was accepted")

    for name in ("fsdp_rmsnorm", "fsdp_rmsnorm_backward", "fsdp_newton_schulz", "fsdp_muon_step"):
        monkeypatch.setattr(fs._lib, name, reached)


def norm(**where):
    at = lambda name: where.get(name, where.get("all", 0))  # noqa: E731
    fs.fsdp_rmsnorm(On(at("x"), 4, 8), On(at("gain"), 8), On(at("y"), 4, 8), residual=On(at("residual"), 4, 8),
                    h_out=On(at("h_out"), 4, 8), rstd=On(at("rstd"), 4, dtype=F32), stream=0)


def backward(**where):
    at = lambda name: where.get(name, where.get("all", 0))  # noqa: E731
    fs.fsdp_rmsnorm_backward(On(at("dy"), 4, 8), On(at("h"), 4, 8), On(at("gain"), 8), On(at("rstd"), 4, dtype=F32),
                             On(at("dx"), 4, 8), On(at("dgain"), 8), On(at("workspace"), 1 << 16, dtype=torch.uint8),
                             dh=On(at("dh"), 4, 8), stream=0)


def newton_schulz(**where):
    at = lambda name: where.get(name, where.get("all", 0))  # noqa: E731
    batch = fs.NewtonSchulzBatch([On(at("source"), 4, 8)], [On(at("out"), 4, 8)])
    fs.fsdp_newton_schulz(batch, On(at("workspace"), 1 << 16, dtype=torch.uint8), stream=0)


def muon(**where):
    at = lambda name: where.get(name, where.get("all", 0))  # noqa: E731
    layout, _ = fs.fsdp_flatten_layout([48, 4], 2)
    state = {k: [On(0, 26, dtype=F32), On(at(k), 26, dtype=F32)] for k in ("master", "exp_avg", "exp_avg_sq")}
    if "all" in where:
        state = {k: [On(where["all"], 26, dtype=F32)] * 2 for k in state}
    unit = fs.MuonUnit(layout, [fs.MuonTensor(8, 6), fs.MuonTensor(4)], [On(at("grads"), 52)] * 2, full_out=On(at("full_out"), 52), **state)
    fs.fsdp_muon_step(unit, fs.Muon(), On(at("workspace"), 1 << 16, dtype=torch.uint8), stream=0)


CALLS = [(norm, ("all", "x", "gain", "y", "residual", "h_out", "rstd")),
         (backward, ("all", "dy", "h", "gain", "rstd", "dx", "dgain", "workspace", "dh")),
         (newton_schulz, ("all", "source", "out", "workspace")),
         (muon, ("all", "grads", "master", "exp_avg", "exp_avg_sq", "full_out", "workspace"))]


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS for n in names], ids=lambda v: getattr(v, "__name__", v))
def test_another_device_is_refused(call, name):
    with pytest.raises(ValueError, match="cuda:1"):
        call(**{name: 1})


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=lambda c: c.__name__)
def test_the_current_device_is_accepted(call):
    with pytest.raises(AssertionError, match="was accepted"):
        call()


def test_a_device_that_is_no_longer_current(monkeypatch):
    batch = fs.NewtonSchulzBatch([On(0, 4, 8)], [On(0, 4, 8)])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0"):
        fs.fsdp_newton_schulz(batch, On(0, 1 << 16, dtype=torch.uint8), stream=0)
