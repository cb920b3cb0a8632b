import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: long-running")


@pytest.fixture(scope="session")
def cuda_device():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _no_collection_between_ranks(request):
    """Ranks of test_sharding_host send tensors by file descriptor and exit after a barrier among themselves, not
    after the parent has fetched them: a collector pass between the parent's gets is long enough to lose that."""
    if request.module.__name__.rpartition(".")[2] != "test_sharding_host":
        yield
        return
    import gc
    gc.collect()
    gc.disable()
    try:
        yield
    finally:
        gc.enable()
