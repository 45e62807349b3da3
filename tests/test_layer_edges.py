"""The layer operators at the edges of what they take: arguments that must be refused before a kernel
sees them, streams given in every form, values that are not finite, states that grow."""
import ctypes

import pytest
import torch

import layer_reference as ref

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qd():
    import delta_rule_linear_qdelta_gb300 as m
    from delta_rule_linear_qdelta_gb300 import build
    build.build()
    m.load_library()
    return m


@pytest.fixture(scope="module")
def layer(qd):
    from delta_rule_linear_qdelta_gb300 import layer as m
    return m


# ------------------------------------------------------------------ workspaces

def test_a_workspace_has_the_memory_that_its_size_says(layer):
    """An expanded tensor has many elements and one byte behind them; a strided one has gaps that are not its own."""
    cpu = torch.device("cpu")
    base = torch.empty(4096, dtype=torch.uint8)
    for bad in (base[:1].expand(4096), base[::2], base.view(64, 64).t()):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            layer._scratch(1024, bad, cpu)
    assert layer._scratch(1024, base, cpu)[:2] == (base.data_ptr(), 4096)
    assert layer._scratch(1024, base.view(torch.float32), cpu)[:2] == (base.data_ptr(), 4096)
