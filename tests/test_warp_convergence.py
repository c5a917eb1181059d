"""Instructions that a whole warp has to run together, by the kernels' sources.

PTX's ``.aligned`` forms (named barriers, cluster barriers, tensor memory) want all lanes of a warp at the
instruction at once; with lanes apart their behaviour is undefined, and a run on a device shows nothing until it
does.  Lanes part in waits that spin lane by lane and in branches of one lane, so what follows one of those needs a
point where the warp meets first.
"""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "sparse_attention_paged_dsa_gb300" / "csrc"
SOURCES = sorted(list(CSRC.glob("*.cu")) + list(CSRC.glob("*.cuh")))

# Barriers and tensor memory's allocation: in wrappers, which meet the warp themselves.
WRAPPED = re.compile(r'"[^"]*(\bbar\.(sync|red)|barrier\.cluster\.\w+[^"]*\.aligned|'
                     r'tcgen05\.(alloc|dealloc|relinquish_alloc_permit)[^"]*\.aligned)')


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
