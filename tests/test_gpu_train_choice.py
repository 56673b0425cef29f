"""Which kernel a product grouped by expert runs on, by its sizes: the names that torch's profiler
reports. The profiled calls run in a process of their own, which leaves this one's launches alone."""
import json
import os
import subprocess
import sys

import pytest
import torch

import block_quantized_moe_gb300 as ft
from test_gpu_train import DEV, check, normal, offsets_of, product_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# (experts, rows, n, k, streaming)
CHOICES = [
    (1, 1, 4096, 7168, True), (1, 4, 1536, 2048, True), (1, 5, 1536, 2048, False), (1, 3, 4096, 7168, False),
    (1, 4, 4096, 7168, False), (1, 16, 512, 1024, False), (2, 2, 1536, 2048, True), (2, 9, 256, 1024, False),
    (8, 8, 512, 7168, True), (8, 8, 1536, 2048, False), (8, 16, 256, 1024, True), (64, 17, 256, 1024, False),
]


def operands(experts, rows, n, k):
    counts = [rows // experts + (e < rows % experts) for e in range(experts)]
    a, w = normal((rows, k), 1.0, torch.bfloat16, 1), normal((experts, n, k), 0.1, torch.bfloat16, 2)
    return counts, a, w, torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)


def profiled():
    """The kernels of one call of each choice, as a JSON line."""
    from torch.profiler import ProfilerActivity, profile
    names = []
    for choice in CHOICES:
        counts, a, w, out = operands(*choice[:4])
        off = offsets_of(counts)
        torch.cuda.synchronize()
        for _ in range(3):  # (a process's first session may report nothing)
            with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
                ft.ftmoe_grouped_matmul(a, off, w, out)
                torch.cuda.synchronize()
            seen = [e.name for e in p.events() if "_kernel<" in e.name]
            if seen:
                break
        names.append(seen)
    print(json.dumps(names))


@pytest.fixture(scope="module")
def names():
    code = f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]; import test_gpu_train_choice as t; t.profiled()"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    got = json.loads(r.stdout.strip().splitlines()[-1])
    if not any(got):
        pytest.skip("the profiler reports no kernels here")
    return got


@pytest.mark.parametrize("i", range(len(CHOICES)))
def test_kernel_choice(i, names):
    streaming = CHOICES[i][4]
    assert len(names[i]) == 1 and ("stream_matmul16" if streaming else "tc_matmul16") in names[i][0], names[i]


@pytest.mark.parametrize("choice", CHOICES)
def test_product_on_either_side_of_the_choice(choice):
    counts, a, w, out = operands(*choice[:4])
    ft.ftmoe_grouped_matmul(a, offsets_of(counts), w, out)
    ref, mag = product_ref(a, w, counts, False)
    check(out, ref, mag, choice[3], "product")
    assert ft.ftmoe_read_error_flags() == 0
