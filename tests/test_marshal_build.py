"""Host check (no GPU): the compiled marshalling module belongs to one Python and
one torch, and is built anew for others."""
import os
import sysconfig

import pytest


def test_marshalling_module_names_the_abis_it_was_built_for(monkeypatch, tmp_path):
    import torch
    import boolean_weight_matmul_b200 as mb
    from boolean_weight_matmul_b200 import build
    here = build.build_marshal()
    assert os.path.exists(here) and torch.__version__ in here and sysconfig.get_config_var("SOABI") in here
    assert build.build_marshal() == here                       # up to date: the same file
    # another torch: the file that is there is neither taken for it nor loaded
    monkeypatch.setattr(torch, "__version__", "99.1+other")
    monkeypatch.setattr(mb, "_marshal_module", None)
    other = build.marshal_path()
    assert other != here and not os.path.exists(other)
    with pytest.raises(RuntimeError, match="is missing; build it"):
        mb._marshal()
    # and building compiles: with the compiler out of reach it fails instead of returning the old file
    monkeypatch.setenv("PATH", str(tmp_path))
    with pytest.raises((FileNotFoundError, RuntimeError)):
        build.build_marshal()
