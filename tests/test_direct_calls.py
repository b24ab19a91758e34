"""The CPython wrappers of the binding beside other threads and where they are missing.  CPU only: the calls end in
stand-ins."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import threading
import time

import pytest

CALLS = {"moe_route_grouped": [1, 1, 64, None, None, 4, 64, 8, 1, 8, 4, 2, 0, 1, 1.0, 1, 1, None],
         "moe_lora": [1, 0, 64, 1, 1, None, None, 1, 1, 1, 1, 16, 4, None, 0, 1, 0, 100, 4, 100, 64, 16, None],
         "moe_combine_norm": [1, 0, 64, 1, 0, None, 1, 0, 0.0, 1e-6, None, 0, 0, 64, 0, 1, 64, 1.0, 1.0, 1, 0, 64, 1, 0, 64, 4,
                              64, None]}


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    """A copy of the wrappers (with variables of its own) whose calls take 0.3 s."""
    from mxfp4_mixture_experts_softmax_gb300 import build_lib
    at = tmp_path_factory.mktemp("direct")
    (at / "slow.c").write_text("#include <time.h>\nint slow(void) { struct timespec t = {0, 300000000}; nanosleep(&t, 0); return 7; }\n")
    subprocess.check_call(["gcc", "-std=gnu11", "-fPIC", "-shared", str(at / "slow.c"), "-o", str(at / "slow.so")])
    copy = str(at / "_pycall.so")
    shutil.copy(build_lib.build_pycall(), copy)
    spec = importlib.util.spec_from_file_location("_pycall", copy)
    direct = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(direct)
    lib = ctypes.CDLL(str(at / "slow.so"))
    for name in CALLS:
        direct.bind(name, ctypes.cast(lib.slow, ctypes.c_void_p).value)
    yield direct
    del lib


@pytest.mark.parametrize("name", CALLS)
def test_other_threads_run_during_a_call(slow, name):
    """A launch may wait for a full queue: Python's lock is not held meanwhile."""
    got = []
    caller = threading.Thread(target=lambda: got.append(getattr(slow, name)(*CALLS[name])))
    caller.start()
    turns = 0
    while caller.is_alive():
        time.sleep(0.005)
        turns += 1
    # 60 turns where the lock is free, one or two where it is held
    assert got == [7] and turns >= 10, turns


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The binding before its first call, with a place for the wrappers where there are none."""
    from mxfp4_mixture_experts_softmax_gb300 import build_lib, libmoe
    build_lib.build()
    monkeypatch.setattr(libmoe, "_lib", None)
    monkeypatch.setattr(build_lib, "PYCALL", str(tmp_path / os.path.basename(build_lib.PYCALL)))
    return libmoe, build_lib


def check_calls(libmoe, lib):
    for name, args in CALLS.items():
        at = len(args) - {"moe_route_grouped": 13, "moe_lora": 5, "moe_combine_norm": 3}[name]
        args = list(args)
        args[at] = 0  # T: nothing to do
        assert getattr(lib, "direct_" + name)(*args) == libmoe.MOE_OK
        args[at] = -1
        assert getattr(lib, "direct_" + name)(*args) == libmoe.MOE_ERR_INVALID_ARG


def test_the_library_loads_without_the_wrappers(fresh):
    libmoe, _ = fresh
    check_calls(libmoe, libmoe.load(build=False))


@pytest.mark.parametrize("left", [b"", b"not a library"])
def test_without_a_compiler(fresh, monkeypatch, left):
    """The built library is used as it is; wrappers of other sources are not."""
    libmoe, build_lib = fresh
    monkeypatch.setenv("CC", "/nonexistent/cc")
    if left:
        with open(build_lib.PYCALL, "wb") as f:
            f.write(left)
        os.utime(build_lib.PYCALL, (1, 1))
    with pytest.warns(RuntimeWarning, match="pycall"):
        lib = libmoe.load()
    assert not os.path.exists(build_lib.PYCALL)
    check_calls(libmoe, lib)


def test_wrappers_that_do_not_load(fresh):
    libmoe, build_lib = fresh
    with open(build_lib.PYCALL, "wb") as f:
        f.write(b"not a library")
    check_calls(libmoe, libmoe.load(build=False))


def test_the_wrappers_name_their_interpreter():
    from mxfp4_mixture_experts_softmax_gb300 import build_lib
    assert build_lib.PYCALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert "cpython" in os.path.basename(build_lib.PYCALL)
