"""Every entry point is among the names that the package gives out."""
import os
import re

import dense_gemm_10_amd as dg
from conftest import ROOT
from dense_gemm_10_amd import grouped, scaled, tokens


def test_every_function_of_the_header_is_exported():
    text = open(os.path.join(ROOT, "include", "densegemm.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(dg_[a-z0-9_]+)\s*\(", text))
    assert len(names) > 15 and names <= set(dg.__all__)


def test_every_torch_entry_point_and_descriptor_is_exported():
    for module in (grouped, tokens, scaled):
        own = {n for n, v in vars(module).items()
               if not n.startswith("_") and getattr(v, "__module__", None) == module.__name__}
        assert own and own <= set(dg.__all__), own - set(dg.__all__)
    assert len(set(dg.__all__)) == len(dg.__all__)
    for name in dg.__all__:
        getattr(dg, name)
