"""Kernels that are launched beside what precedes them in the stream (programmatic dependent launch), by their
sources: what such a kernel must not do shows in no result on the machines where it happens to go well."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "paged_kv_cache_83_gb300" / "csrc"
WAIT = "griddepcontrol.wait"


def code(path):
    """The file without its comments, with the headers of the folder that it includes."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)
    return text + "".join(code(CSRC / name) for name in re.findall(r'#include "([\w.]+)"', text) if name != "pa_common.cuh")


DEPENDENT = [p for p in sorted(CSRC.glob("*.cu")) if WAIT in p.read_text()]


def test_there_are_such_kernels():
    assert {p.name for p in DEPENDENT} >= {"chunk_attn.cu", "chunk_attn_narrow.cu", "decode.cu", "decode_short.cu", "stage.cu"}


@pytest.mark.parametrize("path", DEPENDENT, ids=lambda p: p.name)
def test_nothing_is_read_through_the_read_only_path(path):
    """It asks for data that nothing writes while the kernel runs; the work before may still write when this starts."""
    assert not re.findall(r"__ldg|ld\.global\.nc|ldg_stream|__restrict__ const int32_t", code(path))


@pytest.mark.parametrize("name", ["chunk_attn.cu", "chunk_attn_narrow.cu"])
def test_no_block_waits_for_another_grid_with_tensor_memory(name):
    """A block takes tensor memory after the wait, and lets dependents start after that. Otherwise one kernel's block
    could hold it while it waits for the kernel before, whose block on the same SM waits for tensor memory."""
    text = (CSRC / name).read_text()
    kernel = text[text.index("__global__"):]
    kernel = kernel[:kernel.index("\n}\n")]
    wait, alloc, start = (kernel.index(s) for s in (WAIT, "tmem_alloc(", "griddepcontrol.launch_dependents"))
    sync = kernel.index("__syncthreads()", alloc)
    assert wait < alloc < sync < start
    assert kernel.count("tmem_alloc(") == kernel.count("griddepcontrol.launch_dependents") == 1
