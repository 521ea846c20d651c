"""The binding's compiled step calls an entry point as the header declares it (CPU: every case ends before a call)."""
import os
import re

import pytest

tp = pytest.importorskip("tensor_transformer_mlp_02_amd")
pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def step():
    m = tp._marshaller()
    if not m:
        pytest.skip("the compiled step is not built here")
    return m


def declared():
    """name -> number of arguments of every entry point in include/tpmlp_block.h that enqueues work."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tpmlp_block.h")).read(), flags=re.S)
    return {n: a.count(",") + 1 for n, a in re.findall(r"^int\s+(tp_\w+)\s*\(([^)]*)\)", text, re.M)}


def test_every_declared_entry_point_is_known_with_its_arguments(step):
    found = declared()
    assert len(found) == 6
    for name, count in found.items():
        # as many as declared and no tensor among them: not called
        assert step.call(name, 1, (None,) * (count - 1), None) is None
        for n in (0, count - 2, count, 40):
            with pytest.raises(TypeError, match=f"{name} takes {count - 1} arguments"):
                step.call(name, 1, (None,) * n, None)


def test_other_names_are_refused(step):
    for name in ("tp_moe_permute", "", None, 7):
        with pytest.raises(TypeError, match="no entry point"):
            step.call(name, 1, (None,) * 4, None)
