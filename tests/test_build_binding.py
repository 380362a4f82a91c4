"""CPU: the extension of the paged-cache calls is built beside the library, never in its
way, and never used with another torch than it was built for."""
import os
import sys

import pytest
import torch

import gated_delta_rule_106_b200 as gdn
from gated_delta_rule_106_b200 import _build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The extension's files in a folder of their own."""
    _build.build()
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(_build, "BINDING_STAMP", str(tmp_path / "_paged.built_for"))
    return tmp_path


def test_library_is_built_where_the_extension_cannot_be(elsewhere, monkeypatch):
    which = _build.shutil.which
    for compiler in ("/bin/false", "/nowhere/g++"):
        monkeypatch.setattr(_build.shutil, "which",
                            lambda name: compiler if name == "g++" else which(name))
        with open(_build.BINDING, "w") as f:      # an older one must not stay
            f.write("of another torch")
        with pytest.warns(RuntimeWarning, match="paged-cache calls will raise"):
            assert _build.build() == gdn.library_path()
        assert not os.path.exists(_build.BINDING)


def fake_compiler(folder):
    """Writes its arguments to the output it is asked for."""
    path = folder / "g++"
    path.write_text('#!/bin/sh\necho "$@" > "$(echo "$@" | sed \'s/.*-o //;s/ .*//\')"\n')
    path.chmod(0o755)
    return str(path)


def test_another_torch_builds_the_extension_again(elsewhere, monkeypatch):
    which, fake = _build.shutil.which, fake_compiler(elsewhere)
    monkeypatch.setattr(_build.shutil, "which", lambda name: fake if name == "g++" else which(name))
    read = lambda: open(_build.BINDING).read()  # noqa: E731
    _build.build()
    assert torch.__version__ in read()
    before = os.stat(_build.BINDING).st_mtime_ns
    _build.build()
    assert os.stat(_build.BINDING).st_mtime_ns == before          # nothing changed
    monkeypatch.setattr(torch, "__version__", "0.1.2+other")
    _build.build()
    assert "0.1.2+other" in read()


def test_an_extension_of_another_torch_is_refused(monkeypatch):
    _build.build()
    monkeypatch.setattr(gdn, "_ext", None)
    assert gdn._binding().built_for == torch.__version__
    monkeypatch.setattr(gdn, "_ext", None)
    monkeypatch.setattr(torch, "__version__", "0.1.2+other")
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(RuntimeError, match="built for torch .*0.1.2"):
        gdn.gdn_page_plan(i(3), i(3), i(3, 4), i(9), i(1), 16, token_capacity=8)
    assert gdn.gdn_version() and sys.modules["gated_delta_rule_106_b200"] is gdn
