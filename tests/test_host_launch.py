"""The host side of the launches over a stand-in for the CUDA runtime (tests/cuda/fake_runtime.cpp): no GPU needed."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from quantized_kv_cache_kvq_gb300 import build as b

    lib = b.build()
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    exe = str(tmp_path_factory.mktemp("fake") / "fake_runtime")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-rdynamic", "-I", os.path.join(cuda, "include"), "-o", exe,
                           os.path.join(HERE, "cuda", "fake_runtime.cpp"), lib, f"-Wl,-rpath,{os.path.dirname(lib)}",
                           f"-Wl,-rpath-link,{os.path.join(cuda, 'lib64')}", "-lpthread"])
    env = dict(os.environ, LD_LIBRARY_PATH=os.pathsep.join([os.path.join(cuda, "lib64"), os.environ.get("LD_LIBRARY_PATH", "")]))
    return lambda *a: subprocess.run([exe, *a], capture_output=True, text=True, timeout=120, env=env)


def test_shared_memory_limits_do_not_depend_on_the_call(fake):
    """A kernel's limit is a setting of the device that all threads share: whoever sets it last must not lower it."""
    r = fake("limits")
    assert r.returncode == 0, r.stdout + r.stderr


def test_first_calls_of_two_threads_leave_every_batch_possible(fake):
    r = fake("threads")
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("sms", [152, 100, 1])
def test_the_appends_grid_is_what_the_device_holds_at_once(fake, sms):
    """A persistent grid of more blocks than are resident would run as two waves, each block of the second with a full share."""
    r = fake("grid", str(sms))
    assert r.returncode == 0, r.stdout + r.stderr
    rows = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert len(rows) == 4
    for dtype, batch, blocks, smem in rows:
        fits = 228 * 1024 // (smem + 4096 + 1024)  # two staged tiles, what the device keeps for itself
        assert blocks % sms == 0 and 1 <= blocks // sms <= fits, (dtype, batch, blocks, fits)
        assert blocks // sms >= min(fits, 4)
