"""The serving operators' compiled call layer belongs to one Python and one torch."""
import os
import subprocess
import sysconfig

import pytest
import torch

from long_context_blockwise_max_b200 import build


@pytest.fixture(scope="module")
def S():
    build.build()
    from long_context_blockwise_max_b200 import serving
    return serving


def test_the_call_layer_is_this_torchs_and_this_pythons(S):
    assert S._ordinary.__file__ == build.call_layer_path() == build.build_call_layer()
    name = os.path.basename(S._ordinary.__file__)
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("which", ["torch", "python"])
def test_another_versions_call_layer_is_not_loaded_but_built_anew(S, monkeypatch, which):
    mine = build.call_layer_path()
    if which == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        get = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda n: ".cpython-399-x86_64-linux-gnu.so" if n == "EXT_SUFFIX" else get(n))
    assert build.call_layer_path() != mine
    with pytest.raises(ImportError, match="is not built; run"):
        S._load_call_layer()
    asked = []

    def compiler(cmd, **kw):
        asked.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "")
    monkeypatch.setattr(subprocess, "run", compiler)
    with pytest.raises(RuntimeError, match="call layer"):
        build.build_call_layer()
    assert len(asked) == 1 and os.path.exists(mine)
