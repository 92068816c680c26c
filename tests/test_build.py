"""The build itself, on a source of one line."""
import os

import pytest

from ultra_bit_weight_amd import build as b


def test_library_without_the_binding(tmp_path, monkeypatch):
    """Without torch's headers or g++ the C ABI's library is built all the same,
    and what is missing is said."""
    (tmp_path / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    out = str(tmp_path / "lib" / "libone.so")
    for name, value in (("CSRC", str(tmp_path)), ("BUILD", str(tmp_path / "obj")), ("SOURCES", ["one.cpp"]), ("LIB", out),
                        ("FILE_FLAGS", {})):
        monkeypatch.setattr(b, name, value)

    def no_torch():
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(b, "build_bind", no_torch)
    with pytest.raises(RuntimeError, match="is built.*_sherry_bind.so.*No module named 'torch'"):
        b.build(out=out)
    assert os.path.exists(out)
