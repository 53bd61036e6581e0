"""Grids launched programmatically are resident while earlier work of the stream still writes their inputs, so none of their
loads may be of the kind that wants memory nobody writes meanwhile (__ldg): their sources load inputs through load_input."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).parent.parent / "paged_attention_fp8_gb300" / "csrc"


def code(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def test_one_helper_loads_inputs():
    helper = re.search(r"T load_input\(const T\* p\) \{(.*?)\n\}", code("internal.h"), re.S).group(1)
    assert re.search(r"if constexpr \(EARLY\) return \*p;\s*else return __ldg\(p\);", helper)


# In prefill.cuh the plans' records alone (copied by the host, never written by a kernel) are loaded by __ldg.
@pytest.mark.parametrize("name,allowed", [("blocks.cu", ""), ("decode.cuh", ""), ("prefill.cuh", r"Item load_item\(.*?\n\}")])
def test_no_input_of_an_early_grid_is_loaded_as_constant(name, allowed):
    text = code(name)
    assert "ProgrammaticStreamSerialization" in text and "griddepcontrol.wait" in text
    if allowed:
        text, n = re.subn(allowed, "", text, flags=re.S)
        assert n == 1
    assert not re.findall(r"__ldg|ld\.global\.nc|load_input<false>", text)


def test_the_pair_kernel_is_not_launched_early():
    """Its page ids are loaded by __ldg: it may not become a programmatic launch as it is."""
    text = code("prefill_pair.cuh")
    assert "ProgrammaticStreamSerialization" not in text or "__ldg" not in text
