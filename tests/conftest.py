import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session", autouse=True)
def step_module():
    """Modules' own fixtures build when the library is missing; this one, when
    only the Python module beside it is."""
    from mla_decode_attention_gb300 import build
    if os.path.exists(os.path.join(build.HERE, build.LIB_NAME)) and not os.path.exists(os.path.join(build.HERE, build._step_module())):
        build.build_step()
