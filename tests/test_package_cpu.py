"""What the package offers by name."""
import importlib
import os

import paged_fp8_kv_decode_gb300 as pkg


def test_every_binding_is_named():
    here = os.path.dirname(pkg.__file__)
    bindings = {f[:-3] for f in os.listdir(here) if f.endswith(".py") and "EXPORTED = (" in open(os.path.join(here, f)).read()}
    assert bindings == {"binding", "latent", "rope"} and bindings <= set(pkg.__all__)
    for name in pkg.__all__:
        assert f"``{name}``" in pkg.__doc__
        importlib.import_module(f"{pkg.__name__}.{name}")
