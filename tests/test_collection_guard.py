"""Tests that pass made-up addresses to the library are not run on a machine
with a GPU, where the calls that are accepted would launch kernels on them."""
import ast
import os
import pathlib

import pytest

torch = pytest.importorskip("torch")

import conftest  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    def __init__(self, name):
        self.path, self.markers = pathlib.Path(HERE) / name, []

    def add_marker(self, m):
        self.markers.append(m.name)


@pytest.mark.parametrize("gpu", [False, True])
def test_skipped_where_there_is_a_gpu(gpu, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = [Item(n) for n in sorted(conftest.MADE_UP_ADDRESSES)] + [Item("test_gpu_clip.py")]
    conftest.pytest_collection_modifyitems(items)
    assert [i.markers for i in items] == [["skip"] if gpu else []] * (len(items) - 1) + [[]]


def test_all_of_them_are_named():
    """A file without the gpu marker whose code holds a whole-number address and a direct call of the library."""
    for name in os.listdir(HERE):
        if not name.startswith("test_") or not name.endswith(".py"):
            continue
        tree = ast.parse(open(os.path.join(HERE, name)).read())
        calls = any(isinstance(n, ast.Attribute) and n.attr == "lib" and isinstance(n.value, ast.Name) and n.value.id == "_abi"
                    for n in ast.walk(tree))
        gpu = any(isinstance(n, ast.Name) and n.id == "pytestmark" for n in ast.walk(tree))
        assert not calls or gpu or name in conftest.MADE_UP_ADDRESSES, name
