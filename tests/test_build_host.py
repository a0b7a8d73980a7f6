"""What counts as built: libgdr.so is, with or without the binding's extension, which belongs to one torch."""
import os

import pytest

from gated_deltanet_gdr_b200 import build as gbuild


@pytest.fixture
def away(monkeypatch, tmp_path):
    """the extension and its stamp are looked for and made elsewhere; the library is the built one"""
    gbuild.build()
    monkeypatch.setattr(gbuild, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(gbuild, "MARSHAL", str(tmp_path / os.path.basename(gbuild.MARSHAL)))
    return tmp_path


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler"])
def test_an_extension_that_does_not_compile_is_reported_and_left_out(away, monkeypatch, cxx):
    monkeypatch.setenv("CXX", cxx)
    with open(gbuild.MARSHAL, "w") as f:
        f.write("of another header")
    assert not gbuild.up_to_date()
    with pytest.warns(UserWarning, match="_marshal"):
        assert gbuild.build() == gbuild.LIB
    assert not os.path.exists(gbuild.MARSHAL)  # the old one may not fit the library
    assert gbuild.up_to_date() and gbuild.build() == gbuild.LIB  # and is not tried again


def test_another_torch_or_source_asks_for_another_extension(away, monkeypatch):
    def compiled():
        with open(gbuild.MARSHAL, "w") as f:
            f.write("")
        return True
    monkeypatch.setattr(gbuild, "_compile_marshal", compiled)
    assert not gbuild.up_to_date()
    assert gbuild.build() == gbuild.LIB and gbuild.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(gbuild.importlib.metadata, "version", lambda name: "0.0.1")
        assert not gbuild.up_to_date()
    assert gbuild.up_to_date()
    other = away / "marshal.cpp"
    other.write_text("// changed")
    monkeypatch.setattr(gbuild, "_marshal_sources", lambda: [str(other)])
    assert not gbuild.up_to_date()
    os.remove(gbuild.MARSHAL)
    gbuild.build()
    assert gbuild.up_to_date() and os.path.exists(gbuild.MARSHAL)
