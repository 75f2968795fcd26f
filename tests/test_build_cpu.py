"""The build's order (nothing is compiled)."""

import os

import pytest

from spectral_split_quantized_amd import build


def test_library_is_built_where_the_extension_cannot_be(monkeypatch, tmp_path):
    """The library needs no torch: a failure against torch's headers leaves it built."""
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "OUT", str(tmp_path / "libmetis.so"))

    def run(cmd, verbose):
        open(cmd[cmd.index("-o") + 1], "w").close()

    def no_headers(verbose=False):
        raise RuntimeError("headers")

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "build_tensors", no_headers)
    with pytest.raises(RuntimeError, match="headers"):
        build.build()
    assert os.path.exists(build.OUT)
