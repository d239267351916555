"""The state space block's Python binding without a GPU: what its autograd
functions and argument checks do before anything reaches the library."""
import os
import subprocess

import pytest
import torch

from bidirectional_masked_linear_gb300 import ssm


def _cube(monkeypatch, name):
    """The autograd function `name` on y = x^3 in place of its kernels, applied to x."""
    if name == "LayerNorm":
        monkeypatch.setattr(ssm, "layernorm_fwd", lambda x, *a, **k: (x ** 3, x[..., 0], x[..., 0]))
        monkeypatch.setattr(ssm, "layernorm_bwd", lambda dy, x, *a, **k: (3 * x * x * dy, None, None))
        return lambda x: ssm.LayerNorm.apply(x, x[0].detach(), None)
    if name == "CausalConv":
        monkeypatch.setattr(ssm, "conv_fwd", lambda x, *a, **k: x ** 3)
        monkeypatch.setattr(ssm, "conv_bwd", lambda dy, x, *a, **k: ssm.ConvGrads(3 * x * x * dy, None, None, None))
        return lambda x: ssm.CausalConv.apply(x, x[0].detach(), None)
    monkeypatch.setattr(ssm, "scan_fwd", lambda u, *a, **k: ssm.ScanOut(u ** 3, None, u.detach()))
    monkeypatch.setattr(ssm, "scan_bwd",
                        lambda do, u, *a, **k: ssm.ScanGrads(3 * u * u * do, *[None] * 8))
    return lambda x: ssm.SelectiveScan.apply(x, *[x.detach()] * 4)


@pytest.mark.parametrize("name", ("LayerNorm", "CausalConv", "SelectiveScan"))
def test_second_derivatives_are_refused(monkeypatch, name):
    """The gradients' kernels have none of their own: a second derivative must not come out without their terms."""
    f = _cube(monkeypatch, name)
    x = torch.tensor([[1.0, 2.0]], requires_grad=True)
    g, = torch.autograd.grad(f(x).sum(), x)
    assert torch.equal(g, 3 * x.detach() ** 2)
    g, = torch.autograd.grad(f(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (g.sum() + (x ** 2).sum()).backward()
    # one that does not need them is not refused
    (g.detach().sum() + (x ** 2).sum()).backward()
    assert torch.equal(x.grad, 2 * x.detach())
    # nor is one with nothing to differentiate
    dy = torch.ones_like(x)
    assert not torch.autograd.grad(f(x), x, dy)[0].requires_grad


class _On:
    """What the checks look at of a tensor on GPU `k`."""
    dtype, is_cuda, shape = torch.float32, True, (2, 4, 8)

    def __init__(self, k):
        self.k, self.device = k, torch.device("cuda", k)

    def get_device(self):
        return self.k


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: tensors of another one must not get that far."""
    monkeypatch.setattr(ssm, "_current_device", lambda: 0)
    monkeypatch.setattr(ssm, "load", lambda: None)
    assert ssm._code(_On(0)) == 1
    x = _On(1)
    for call in (lambda: ssm._code(x), lambda: ssm.layernorm_fwd(x, x), lambda: ssm.layernorm_bwd(x, x, x, x, x),
                 lambda: ssm.conv_fwd(x, x), lambda: ssm.conv_bwd(x, x, x), lambda: ssm.conv_step(x, x, x),
                 lambda: ssm.scan_fwd(x, x, x, x, x), lambda: ssm.scan_bwd(x, x, x, x, x, x),
                 lambda: ssm.scan_step(x, x, x, x, x, x)):
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            call()

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ssm._handle(Stream, _On(0))
    assert ssm._handle(Stream, x) == 7


def test_memory_that_a_device_can_use(tmp_path):
    """The library's own check of every pointer (ssm_check.h): another device's memory is refused."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "check.cpp"
    src.write_text(
        '#include <cstdio>\n#include <initializer_list>\n#include "ssm_check.h"\n'
        "int main() {\n"
        "  for (int type : {cudaMemoryTypeUnregistered, cudaMemoryTypeHost, cudaMemoryTypeDevice,"
        " cudaMemoryTypeManaged})\n"
        "    for (int device = 0; device < 2; ++device) for (int mapped = 0; mapped < 2; ++mapped) {\n"
        "      cudaPointerAttributes at = {};\n"
        "      at.type = (cudaMemoryType)type; at.device = device;\n"
        "      at.devicePointer = mapped ? &at : nullptr;\n"
        '      printf("%d", (int)lion::usable_on(at, 1));\n'
        "    }\n"
        "}\n")
    exe = tmp_path / "check"
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(root, "bidirectional_masked_linear_gb300", "csrc"),
                    "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    # (device 0 unmapped, mapped; device 1 unmapped, mapped) of each kind
    assert got == "0000" "0101" "0011" "1111"


def test_token_counts_near_32_bits_are_refused():
    """Past LION_SSM_MAX_EXTENT an index plus a segment's length would not fit an int."""
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())
    most = 2 ** 31 - 2 ** 16
    for L, taken in ((most, True), (most + 1, False), (2 ** 31 - 1, False)):
        assert (ssm.conv_bwd_workspace_bytes(1, L, 8, 4) > 0) is taken
        assert (ssm.scan_workspace_bytes(1, L, 8, 16) > 0) is taken
        assert (ssm.scan_bwd_workspace_bytes(1, L, 8, 16) > 0) is taken


def test_channel_counts_near_32_bits_are_refused():
    """Past LION_SSM_MAX_EXTENT a channel's place, or that of a group's row of B, would not fit an int."""
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())
    most = 2 ** 31 - 2 ** 16
    for D, taken in ((most, True), (most + 1, False), (2 ** 31 - 2, False)):
        assert (ssm.conv_bwd_workspace_bytes(1, 1, D, 4) > 0) is taken
        assert (ssm.scan_bwd_workspace_bytes(1, 1, D, 8) > 0) is taken
    assert ssm.scan_bwd_workspace_bytes(1, 1, 2 ** 24, 64, 2 ** 24) > 0
    assert ssm.scan_bwd_workspace_bytes(1, 1, 2 ** 25, 64, 2 ** 25) == 0


def test_workspace_counts_bytes_that_it_has():
    """An expanded tensor has more elements than memory behind them."""
    ws = torch.zeros(64, dtype=torch.uint8)
    assert ssm._workspace(ws, None, None, "scan") == (ws.data_ptr(), 64, ws)
    for bad in (ws[:1].expand(4096), ws.view(8, 8).t(), ws[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            ssm._workspace(bad, None, None, "scan")
