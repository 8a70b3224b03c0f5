"""What the binding of the cache's operators refuses before it looks at anything else, on
the host."""
import os

import pytest
import torch

import w8a8_int8_expert_amd as m


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(m.LIB_PATH):
        from w8a8_int8_expert_amd import build
        build.build()
    return m.load_library()


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("bad", [None, 5, [5], (0, 1), "5", [[1]]])
def test_batches_of_what_is_no_tensor(which, bad):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    a = [z(2), z(1), z(1, 4)]
    a[which] = bad
    with pytest.raises(m.MoEW8A8Error):
        m.SequenceBatch(*a, 1, 9)
