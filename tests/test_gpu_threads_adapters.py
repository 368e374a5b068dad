"""The balance loss and the adapters from threads at once: what goes wrong in a thread fails the test."""

from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from test_gpu_adapters_and_balance import SIZES, batch, everything

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def test_threads_at_once():
    cases = []
    for i, size in enumerate(SIZES):
        d, cut = batch(*size, seed=20 + i)
        cases.append((d, cut, size[2], M.LoRAAdapters(d["down"], d["up"], d["scale"])))
    want = [everything(*c) for c in cases]
    torch.cuda.synchronize()

    def run(i):
        same = 0
        with torch.cuda.stream(torch.cuda.Stream()):
            for turn in range(6):
                at = (i + turn) % len(cases)
                got = everything(*cases[at])
                torch.cuda.current_stream().synchronize()
                same += all(torch.equal(a, b) for a, b in zip(got, want[at], strict=True))
        return same

    with ThreadPoolExecutor(8) as pool:
        assert [f.result() for f in [pool.submit(run, i) for i in range(8)]] == [6] * 8
    assert M.nvfp4_get_device_error() == 0
