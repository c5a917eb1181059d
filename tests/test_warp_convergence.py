"""Instructions that a whole warp has to run together, by the kernels' sources.

PTX's ``.aligned`` forms (named barriers, cluster barriers, tensor memory) want all lanes of a warp at the
instruction at once; with lanes apart their behaviour is undefined, and a run on a device shows nothing until it
does.  Lanes part in waits that spin lane by lane and in branches of one lane, so what follows one of those needs a
point where the warp meets first.
"""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "sparse_attention_paged_dsa_gb300" / "csrc"
SOURCES = sorted(list(CSRC.glob("*.cu")) + list(CSRC.glob("*.cuh")))

# Barriers and tensor memory's allocation: in wrappers, which meet the warp themselves.
WRAPPED = re.compile(r'"[^"]*(\bbar\.(sync|red)|barrier\.cluster\.\w+[^"]*\.aligned|'
                     r'tcgen05\.(alloc|dealloc|relinquish_alloc_permit)[^"]*\.aligned)')
# In the kernels' loops: reads and writes of tensor memory.
ALIGNED = re.compile(r"\b(tmem_(ld|st)_\w+|stmatrix_\w+)\(")
MEET = re.compile(r"__syncwarp\(|__syncthreads\w*\(|__(all|any|ballot|shfl\w*|reduce_\w+)_?sync\(|"
                  r"\b(soft_or|soft_bar_or|soft_bar_sync|softmax_bar_or|softmax_bar_sync|cluster_sync_all|quad_sync)\(")
# (`wait(...)`: the kernels' own wrappers around a wait, which vote)
PART = re.compile(r"\bmbar_(await|wait|wait_cluster)\(|\bwait_landed\w*\(|\bif \(lane|\bif \(threadIdx|\bif \(need\)|"
                  r"\bif \(head_thr\)|live_row|\balpha = exp2f|flagged = true|\bissuer\)")


def code(path):
    """The lines of a file without comments."""
    text = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), path.read_text(), flags=re.S)
    return [re.sub(r"//.*", "", line) for line in text.splitlines()]


def test_barrier_wrappers_meet_the_warp():
    """Each wrapper of an aligned barrier starts with a point where the warp meets."""
    seen = 0
    for path in SOURCES:
        lines = code(path)
        for n, line in enumerate(lines):
            if not WRAPPED.search(line):
                continue
            seen += 1
            start = max(i for i in range(n + 1) if re.match(r"(template|__device__)", lines[i]))
            assert "__device__ __forceinline__" in lines[start], f"{path.name}:{n + 1}: not in a wrapper"
            body = "\n".join(lines[start:n + 1])
            assert "__syncwarp();" in body.split("asm")[0], f"{path.name}:{n + 1}: lanes may be apart"
    assert seen >= 10


@pytest.mark.parametrize("path", [p for p in SOURCES if p.suffix == ".cu"], ids=lambda p: p.name)
def test_tensor_memory_is_read_by_whole_warps(path):
    """Between a place where lanes may part and a read or write of tensor memory the warp meets."""
    lines = code(path)
    for n, line in enumerate(lines):
        if not ALIGNED.search(line) or "__device__" in line:
            continue
        for i in range(n - 1, -1, -1):
            if MEET.search(lines[i]) or ALIGNED.search(lines[i]):
                break
            assert not PART.search(lines[i]), f"{path.name}:{n + 1}: lanes may be apart since line {i + 1}"
