"""A binding built for another torch or Python is neither loaded nor taken as built."""
import os
import sysconfig

import torch

from paged_mla_decode_07_gb300 import builder


def test_the_binding_belongs_to_one_torch_and_one_python(monkeypatch):
    builder.build()
    assert builder.BINDING == builder.binding_path() and os.path.exists(builder.BINDING) and builder.binding_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0+other")
        m.setattr(builder, "BINDING", builder.binding_path())
        assert not builder.binding_up_to_date() and builder.library_up_to_date()
    soabi = sysconfig.get_config_var("SOABI")
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-39-other" if name == "SOABI" else None)
        assert builder.binding_path() != builder.BINDING
    assert soabi in builder.BINDING and torch.__version__ in builder.BINDING
