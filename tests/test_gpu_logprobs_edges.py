"""gem_logprobs at the edges of its call: infinite tokens, the least and largest scales, arguments it has no use for."""
import numpy as np
import pytest

from oracle import fp8
from test_gpu_logprobs import _check, _logits, _run, env  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_workspace_may_be_given(env):  # noqa: F811
    """Calls that pass one, as the other calls with scratch take it, give what calls without one give."""
    gem, t = env
    y = _logits(5, 9001, 1)
    scratch = t.empty(1 << 20, dtype=t.uint8, device="cuda")
    scratch.fill_(0xA5)
    a, b = _run(env, y, [0, 1, 2, 3, 9000], 7), _run(env, y, [0, 1, 2, 3, 9000], 7, workspace=scratch)
    assert all(np.array_equal(a[n], b[n]) for n in a)
    assert bool((scratch == 0xA5).all())
    for bad in (scratch.float(), scratch.cpu(), scratch[::2]):
        with pytest.raises(ValueError):
            _run(env, y, [0, 1, 2, 3, 4], 7, workspace=bad)
