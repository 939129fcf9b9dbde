"""Walks over so many states that a unit takes longer than the limit of a wait
(2 s by default, more than 100 million states; 1 ms here, in a child process,
since the limit is read once): nothing gives up, and the results are right."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from context_attention_long_b200 import api, build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def check_long_walk(units):
    """`units` pairs of query tiles (as many as SMs: a walk each; one: shared by
    a cluster) against 400000 states, 3125 steps of some 2 us, or 1600000, half of that each."""
    from test_gpu_cross import check_forward, normal
    Sq, Skv, D = 256 * units, 400000 if units > 1 else 1600000, 64
    q, k, v = normal(1, Sq, 1, D, seed=1), normal(1, Skv, 1, D, seed=2), normal(1, Skv, 1, D, seed=3)
    out, lse = api.cpattn_cross_attention(q, k, v)
    assert api.cpattn_device_status() == (0, 0)
    check_forward(q, k, v, None, out, lse, np.unique(np.linspace(0, Sq - 1, 7).astype(int)))


@pytest.mark.parametrize("shared", [False, True])
def test_a_walk_longer_than_the_limit(shared):
    units = 1 if shared else torch.cuda.get_device_properties(0).multi_processor_count
    code = f"import test_gpu_cross_wait_limits as t; t.check_long_walk({units})"
    env = dict(os.environ, CPATTN_WAIT_TIMEOUT_MS="1",
               PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE), os.environ.get("PYTHONPATH", "")]))
    done = subprocess.run([sys.executable, "-c", code], env=env, cwd=HERE, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stdout + done.stderr
