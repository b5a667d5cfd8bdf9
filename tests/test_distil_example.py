"""The operators together, as examples/distil_head.py uses them: the student learns."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,vocab", [(200, 256, 5000), (9, 128, 1003)])
def test_student_learns(tokens, hidden, vocab):
    spec = importlib.util.spec_from_file_location("distil_head",
                                                  os.path.join(ROOT, "examples", "distil_head.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    seen = mod.run(tokens, hidden, vocab, 8, log=lambda *_: None)
    assert all(b > a for a, b in zip(seen, seen[1:]))
    assert seen[-1] > seen[0] + 1.0
