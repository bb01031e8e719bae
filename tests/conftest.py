import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# The binding works without its compiled marshalling; that module's own tests need it to be imported.
try:
    from bit_weight_only_w2_b200 import _marshal  # noqa: F401
    collect_ignore = []
except ImportError:
    collect_ignore = ["test_marshal.py"]


def pytest_report_header(config):
    return [f"left out, no _marshal.so for this PyTorch: {name}" for name in collect_ignore]


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU and the built CUDA library")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device in this process")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
