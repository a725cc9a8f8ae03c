"""When a build is out of date: any source newer than what was built from it."""
import os

import pytest

from dense_gemm_14_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Sources and built files of one age, in place of the repository's."""
    made = {}
    for name, paths in (("SOURCES", build.SOURCES), ("HEADERS", build.HEADERS), ("LIB_PATH", [build.LIB_PATH]),
                        ("MARSHAL_SOURCE", [build.MARSHAL_SOURCE]), ("MARSHAL_PATH", [build.MARSHAL_PATH])):
        made[name] = [str(tmp_path / os.path.basename(p)) for p in paths]
        for p in made[name]:
            open(p, "w").close()
            os.utime(p, (1000, 1000))
        monkeypatch.setattr(build, name, made[name] if name in ("SOURCES", "HEADERS") else made[name][0])
    return made


def test_one_age_is_not_stale(tree):
    assert not build.stale()


@pytest.mark.parametrize("name", ["SOURCES", "HEADERS", "MARSHAL_SOURCE"])
def test_a_newer_source_is_stale(tree, name):
    for p in tree[name]:
        os.utime(p, (2000, 2000))
        assert build.stale(), p
        os.utime(p, (1000, 1000))


@pytest.mark.parametrize("name", ["LIB_PATH", "MARSHAL_PATH"])
def test_a_missing_file_is_stale_and_each_is_compared_with_its_own(tree, name):
    os.utime(tree["MARSHAL_SOURCE"][0], (1500, 1500))
    os.utime(tree["LIB_PATH"][0], (2000, 2000))
    assert build.stale()                  # the library's age says nothing about the marshalling's
    os.utime(tree["MARSHAL_PATH"][0], (2000, 2000))
    assert not build.stale()
    os.remove(tree[name][0])
    assert build.stale()
