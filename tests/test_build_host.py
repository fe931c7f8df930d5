"""The build looks at every file that the library is made of."""
import os

from dense_gemm_engineering_bf16_b200 import build as B


def files(*folders):
    return {os.path.join(f, n) for f in folders for n in os.listdir(f) if os.path.isfile(os.path.join(f, n))}


def test_every_source_and_header_is_a_dependency():
    assert set(B._deps()) == files(B.CSRC, B.INCLUDE)


def test_an_edit_of_any_file_asks_for_a_build(monkeypatch):
    """Each file in turn is made to look newer than the library."""
    real = os.path.getmtime
    built = 2.0e9
    for edited in sorted(files(B.CSRC, B.INCLUDE)):
        times = {B.LIB: built, edited: built + 1}
        monkeypatch.setattr(B.os.path, "exists", lambda p: True)
        monkeypatch.setattr(B.os.path, "getmtime", lambda p: times.get(p, built - 1))
        assert B.needs_build(), edited
        times[edited] = built - 1
        assert not B.needs_build()
        monkeypatch.setattr(B.os.path, "getmtime", real)
