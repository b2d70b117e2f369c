import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Host-side tests that also make calls which are not refused, with addresses that are no memory: without a
# device these stop before the launch.
NO_DEVICE = ("test_qk_norm_rope_refusals", "test_cache_write_refusals")


def pytest_collection_modifyitems(items):
    mine = [i for i in items if i.name in NO_DEVICE]
    if not mine:
        return
    import torch
    if torch.cuda.is_available():
        for i in mine:
            i.add_marker(pytest.mark.skip(reason="would launch kernels on addresses that are no memory"))


# Mismatch counts of the one-ulp parity checks (LayerNorm y, QKV-epilogue q and k: elements
# that differ from the oracle by one bf16 ulp), reported at the end of the run.
PARITY_COUNTS = []


def pytest_terminal_summary(terminalreporter):
    if not PARITY_COUNTS:
        return
    total = sum(n for _, n, _ in PARITY_COUNTS)
    elems = sum(e for _, _, e in PARITY_COUNTS)
    terminalreporter.write_line(
        f"one-ulp parity (LayerNorm y, QKV q/k): {len(PARITY_COUNTS)} checks, {elems} elements, "
        f"{total} differ from the oracle by 1 bf16 ulp (none by more)")
    for what, n, e in PARITY_COUNTS:
        if n:
            terminalreporter.write_line(f"  {what}: {n} of {e}")
