import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs the sm_103a kernels)")
    config.addinivalue_line("markers", "slow: full-size workload")


@pytest.fixture(autouse=True)
def _binding_as_loaded(request, monkeypatch):
    """Tests without a GPU see the binding as it is before its first call, which looks up torch's calls for
    streams and memory: what a call on a GPU left there does not reach those that stand in for the library."""
    if "gpu" not in request.keywords:
        from int8_paged_kv_gb300 import _binding
        for name in ("_current_device", "_raw_stream", "_raw_alloc", "_raw_delete"):
            monkeypatch.setattr(_binding, name, None)
        monkeypatch.setattr(_binding, "_U32", ())
    yield


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle
    oracle.build()
    return oracle
