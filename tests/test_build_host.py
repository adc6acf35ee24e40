"""What build() takes for out of date: an object is compared with the files it
was compiled from, whatever has become of the list beside it."""
import os

import pytest

from microscaling_quantized_convolution_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one source and two headers, its object the newest."""
    csrc, inc = tmp_path / "pkg" / "csrc", tmp_path / "include"
    csrc.mkdir(parents=True)
    inc.mkdir()
    monkeypatch.setattr(B, "ROOT", str(tmp_path))
    monkeypatch.setattr(B, "CSRC", str(csrc))
    for i, f in enumerate((csrc / "a.cu", csrc / "used.cuh", csrc / "other.cuh", inc / "mqv.h", csrc / "a.o")):
        f.write_text("")
        os.utime(f, (1000 + i, 1000 + i))
    return csrc


def _listed(csrc, root, names=("a.cu", "used.cuh")):
    (csrc / "a.d").write_text(f"{root}/a.o : " + " \\\n  ".join(f"{root}/{n}" for n in names) + "\n")


def _stale(csrc):
    return B._stale(str(csrc / "a.o"), B._object_deps("a.cu"))


def test_object_is_compared_with_its_own_files(tree):
    _listed(tree, tree)
    assert not _stale(tree)
    os.utime(tree / "other.cuh", (2000, 2000))
    assert not _stale(tree)
    os.utime(tree / "used.cuh", (2000, 2000))
    assert _stale(tree)


def test_a_list_with_a_missing_file_is_out_of_date(tree):
    _listed(tree, tree, ("a.cu", "used.cuh", "gone.cuh"))
    assert _stale(tree)


def test_a_copied_tree_does_not_trust_the_list_of_the_first(tree):
    """The list names the place that the tree was built in; in a copy of the
    tree every header counts, or a changed source would be left uncompiled."""
    _listed(tree, "/elsewhere/pkg/csrc")
    assert not _stale(tree)
    os.utime(tree / "a.cu", (2000, 2000))
    assert _stale(tree)


@pytest.mark.parametrize("text", ["", "a.o", "a.o :"])
def test_a_cut_off_list_is_as_good_as_none(tree, text):
    (tree / "a.d").write_text(text)
    assert not _stale(tree)
    os.utime(tree / "used.cuh", (2000, 2000))
    assert _stale(tree)
