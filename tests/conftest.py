import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU case")


def pytest_sessionstart(session):
    """A tree whose library was built before the tensor binding existed is built again (where it can be: without
    the binding the training operators' tests say what is missing)."""
    import importlib.util

    from matrix_dense_linear_spd_gb300 import build
    if os.path.exists(build.LIB) and not os.path.exists(build.BINDING) and importlib.util.find_spec("torch"):
        try:
            build.build()
        except (RuntimeError, OSError) as e:
            print(f"the tensor binding could not be built: {e}", file=sys.stderr)
