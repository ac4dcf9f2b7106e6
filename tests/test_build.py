"""Which built files are taken as they are (CPU)."""
import torch

from bit_nf4_quantized_quant_b200 import build


def test_binding_of_another_torch_is_stale(monkeypatch):
    """The binding is linked to torch's C++ libraries: one that another torch was there for is built again."""
    build.build()
    assert not build._binding_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build._binding_stale()
