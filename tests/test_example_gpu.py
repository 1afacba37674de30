"""The example that runs the operators around a replay buffer: the drafter learns."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_drafter_learns_from_replay():
    from rl_infra_gb300 import build, capi
    build.build()
    capi.load()
    spec = importlib.util.spec_from_file_location("draft_replay", os.path.join(ROOT, "examples", "draft_replay.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last = example.main(rounds=150, seed=0, say=None)
    # an untrained draft is accepted by chance; a trained one clearly more often
    assert last > first + 0.1
