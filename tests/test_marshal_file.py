"""The compiled marshalling belongs to one interpreter: its file carries that
interpreter's tag, so that another builds its own instead of loading this one."""
import os
import subprocess
import sys
import sysconfig

import dense_gemm_14_amd
from dense_gemm_14_amd import build


def test_the_file_carries_the_interpreters_tag():
    assert os.path.basename(build.MARSHAL_PATH) == "_marshal" + sysconfig.get_config_var("EXT_SUFFIX")
    assert sysconfig.get_config_var("SOABI") in build.MARSHAL_PATH


def test_the_package_imports_that_file():
    dense_gemm_14_amd.load()
    if not os.path.exists(build.MARSHAL_PATH):
        build.build_marshal()
    p = subprocess.run([sys.executable, "-c", "from dense_gemm_14_amd import _marshal; print(_marshal.__file__)"],
                       cwd=build.ROOT, capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and os.path.samefile(p.stdout.strip(), build.MARSHAL_PATH), p.stdout + p.stderr
