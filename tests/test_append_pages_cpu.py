"""The append's page lookup for any numbers that its tables can hold (run on the host, no GPU needed)."""
import os
import shutil
import subprocess

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))


def lookup(tmp_path, cases):
    exe = str(tmp_path / "page_of_run")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.check_call([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-o", exe, os.path.join(HERE, "cuda", "page_of_run.cu")])
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_a_page_is_one_of_the_runs_or_none(tmp_path):
    rng = np.random.default_rng(1)
    top = 1 << 30  # the longest context
    firsts = [0, 1, 15, 16, 17, 100, top - 1, -1, -15, -16, -17, -1000, -top]
    lens = [0, 1, 16, 17, 33, 100, 2000, top]
    nths = [0, 1, 2, 5, 100, -1, -3, 1 << 26, (1 << 26) - 1]
    cases = [(f, n, i) for f in firsts for n in lens for i in nths]
    cases += [tuple(int(v) for v in (rng.integers(-200, 200), rng.integers(0, 200), rng.integers(-5, 20))) for _ in range(3000)]
    real = 0
    for (first, n, nth), (f, p0, start, end, page) in zip(cases, lookup(tmp_path, cases), strict=True):
        pages = range(first // 16, (n - 1) // 16 + 1) if 0 <= first < n else range(0)
        if 0 <= nth < len(pages):
            want = pages[nth]
            assert (f, page, p0, start, end) == (first, want, 16 * want, max(first - 16 * want, 0), min(n - 16 * want, 16))
            real += 1
        else:  # its table entry is read all the same
            assert end <= start and 0 <= page <= (max(n, 1) - 1) // 16, (first, n, nth)
    assert real > 200
