"""The torch binding of the router, the expert layer and the orthogonalisation over several devices, without a GPU: the
real source over fake devices (tests/fake_devices), as in test_operators_device.py."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sysconfig

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    root, lib = os.path.dirname(HERE), os.path.join(os.path.dirname(torch.__file__), "lib")
    include = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    out = str(tmp_path_factory.mktemp("fake") / "_sar_torch.so")
    run = subprocess.run(
        ["g++", "-O0", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w", "-I", os.path.join(HERE, "fake_devices"),
         "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"], "-I", include,
         "-I", os.path.join(include, "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
         os.path.join(HERE, "fake_devices", "binding_block.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
         "-Wl,-rpath," + lib], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-4000:]
    spec = importlib.util.spec_from_file_location("_sar_torch", out)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.c = ctypes.PyDLL(out)
    module.c.fake_tensor.restype, module.c.fake_tensor.argtypes = ctypes.py_object, [ctypes.py_object, ctypes.c_int]
    module.c.fake_stream.restype = ctypes.c_size_t
    module.host = []                                   # what the fake tensors lie in
    return module


def calls(fake, device):
    def on(*shape, dtype=torch.float32):
        fake.host.append(torch.zeros(*shape, dtype=dtype))
        return fake.c.fake_tensor(fake.host[-1], device)
    x, ids, w = on(4, 8), on(4, 2, dtype=torch.int32), on(4, 2)
    return {
        "route": lambda **k: fake.sar_expert_route(x, ids, w, **k),
        "route_backward": lambda **k: fake.sar_expert_route_backward(w, x, ids, on(4, 8), **k),
        "layer": lambda **k: fake.sar_expert_layer(x, ids, on(3, 12, 8), on(3, 8, 6), on(4, 8), w, workspace=on(64), **k),
        "orthogonalize": lambda **k: fake.sar_orthogonalize(on(2, 4, 8), on(2, 4, 8), on(64), **k),
    }


NAMES = ["route", "route_backward", "layer", "orthogonalize"]


class Stream:
    def __init__(self, device, handle):
        self.device_index, self.cuda_stream = device, handle


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current,device", [(0, 0), (0, 1), (1, 0), (2, 1)])
def test_calls_run_on_the_tensors_device(fake, name, current, device):
    fake.c.fake_current(current)
    before = fake.c.fake_calls()
    calls(fake, device)[name]()
    assert fake.c.fake_calls() == before + 1
    assert fake.c.fake_device() == device and fake.c.fake_stream() == 0x1000 + device
    assert fake.c.fake_current(-1) == current


@pytest.mark.parametrize("name", NAMES)
def test_refused_calls_leave_the_current_device(fake, name):
    fake.c.fake_current(0)
    before = fake.c.fake_calls()
    with pytest.raises(AttributeError):
        calls(fake, 1)[name](stream=object())
    with pytest.raises(ValueError):
        calls(fake, 1)[name](stream=Stream(0, 0x77))
    assert fake.c.fake_calls() == before and fake.c.fake_current(-1) == 0
    calls(fake, 1)[name](stream=Stream(1, 0x77))
    assert fake.c.fake_device() == 1 and fake.c.fake_stream() == 0x77


def test_tensors_of_two_devices_are_refused(fake):
    def on(device, *shape, dtype=torch.float32):
        fake.host.append(torch.zeros(*shape, dtype=dtype))
        return fake.c.fake_tensor(fake.host[-1], device)
    for call in (lambda: fake.sar_expert_route(on(0, 4, 8), on(1, 4, 2, dtype=torch.int32), on(0, 4, 2)),
                 lambda: fake.sar_expert_layer(on(0, 4, 8), on(0, 4, 2, dtype=torch.int32), on(0, 3, 12, 8), on(1, 3, 8, 6), on(0, 4, 8)),
                 lambda: fake.sar_orthogonalize(on(0, 4, 8), on(0, 4, 8), on(1, 64))):
        with pytest.raises(ValueError):
            call()
