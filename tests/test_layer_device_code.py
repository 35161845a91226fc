"""The machine code of the kernels between token ids and the expert layer: the wait states
that inline assembly needs, nothing in scratch memory, no packed fp32 arithmetic."""
import pytest

from test_device_code import disassembly, hazards

SOURCES = ["nsg_embed.hip", "nsg_norm.hip", "nsg_route.hip"]


@pytest.mark.parametrize("source", SOURCES)
def test_layer_device_code(source, tmp_path):
    functions = disassembly(source, tmp_path)
    assert not [(f"{a:x}", w) for f in functions for a, w in hazards(f)]
    names = {name for f in functions for name, _, _ in f}
    assert not [n for n in names if n.startswith("scratch_") or n in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")]
