"""The torch binding over several devices, without a GPU: the real source over
fake devices and a library that records the device that is current at each call
(tests/fake_devices).  The calls go to the tensors' device, whichever is
current, and the current device is as before when they return or raise."""
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
         os.path.join(HERE, "fake_devices", "binding.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
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
    """Each operator's call over tensors of a fake device, taking more keyword arguments."""
    def on(*shape, dtype=torch.float32):
        fake.host.append(torch.zeros(*shape, dtype=dtype))
        return fake.c.fake_tensor(fake.host[-1], device)
    i32 = dict(dtype=torch.int32)
    x, y, f, pos = on(4, 8), on(4, 8), on(4), on(4, 2, **i32)
    rows, w = on(8, 8), on(4, 2)
    return {
        "layer_norm": lambda **k: fake.sar_layer_norm(x, y, **k),
        "layer_norm_backward": lambda **k: fake.sar_layer_norm_backward(x, x, None, f, f, y, **k),
        "sort": lambda **k: fake.sar_expert_sort(pos, on(3, **i32), on(4, **i32), on(4, 2, **i32), **k),
        "dispatch": lambda **k: fake.sar_expert_dispatch(x, pos, rows, **k),
        "combine": lambda **k: fake.sar_expert_combine(rows, pos, y, **k),
        "combine_backward": lambda **k: fake.sar_expert_combine_backward(x, rows, pos, w, rows, **k),
    }


NAMES = ["layer_norm", "layer_norm_backward", "sort", "dispatch", "combine", "combine_backward"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current,device", [(0, 0), (0, 1), (1, 0), (2, 1)])
def test_calls_run_on_the_tensors_device(fake, name, current, device):
    fake.c.fake_current(current)
    before = fake.c.fake_calls()
    calls(fake, device)[name]()
    assert fake.c.fake_calls() == before + 1
    assert fake.c.fake_device() == device and fake.c.fake_stream() == 0x1000 + device
    assert fake.c.fake_current(-1) == current
    calls(fake, device)[name](stream=0)                 # the default stream is the current device's
    assert fake.c.fake_device() == device and fake.c.fake_stream() == 0
    assert fake.c.fake_current(-1) == current


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_call_leaves_the_current_device(fake, name):
    fake.c.fake_current(0)
    before = fake.c.fake_calls()
    with pytest.raises(AttributeError):
        calls(fake, 1)[name](stream=object())
    assert fake.c.fake_calls() == before and fake.c.fake_current(-1) == 0


class Stream:
    def __init__(self, device, handle):
        self.device_index, self.cuda_stream = device, handle


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(fake, name):
    fake.c.fake_current(0)
    calls(fake, 1)[name](stream=Stream(1, 0x77))
    assert fake.c.fake_device() == 1 and fake.c.fake_stream() == 0x77
    before = fake.c.fake_calls()
    with pytest.raises(ValueError):
        calls(fake, 1)[name](stream=Stream(0, 0x77))
    assert fake.c.fake_calls() == before and fake.c.fake_current(-1) == 0
