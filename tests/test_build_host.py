"""The order of the build, without compiling the library: the C library does not wait for what needs torch's headers."""
import os

import pytest

from convolution_forward_conv2d_amd import build


def test_the_library_does_not_need_the_binding(tmp_path, monkeypatch):
    (tmp_path / "one.cpp").write_text('extern "C" int one() { return 1; }\n')

    def no_headers(verbose):
        raise RuntimeError("g++ failed on binding.cpp: no torch headers")

    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", ["one.cpp"])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_one.so"))
    monkeypatch.setattr(build, "_compile_binding", no_headers)
    with pytest.raises(RuntimeError, match="torch headers"):               # said, not passed over
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.NATIVE)
