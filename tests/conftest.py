import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long CPU test, deselect with -m 'not slow'")


def pytest_collection_modifyitems(config, items):
    # GPU tests fail loudly when no GPU is present rather than silently passing; they are
    # deselected on CPU-only hosts with -m "not gpu".
    pass


# Tests that give work to a new stream while their inputs are still being filled on the current one.
STREAMS_START_BEHIND = {"test_llama7b_layers_from_eight_shards_full_size"}


@pytest.fixture(autouse=True)
def _streams_start_behind(request, monkeypatch):
    """Lets every stream that such a test makes wait for what the current stream has been given by then, so that its result
    does not hang on how long the fill takes, and so on which tests ran before."""
    if request.node.name not in STREAMS_START_BEHIND:
        return
    import torch
    make = torch.cuda.Stream

    def behind(*args, **kw):
        stream = make(*args, **kw)
        if not args and not kw:  # torch makes handles of streams that exist with their ids
            stream.wait_stream(torch.cuda.current_stream())
        return stream

    monkeypatch.setattr(torch.cuda, "Stream", behind)
