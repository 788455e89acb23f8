"""Rules that the kernels' sources keep and that no result shows."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_sort_amd", "csrc")


def _sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*", "", f.read())


def _calls(text, name):
    """Argument lists (top-level commas) of the calls of `name`."""
    for m in re.finditer(re.escape(name) + r"\s*\(", text):
        args, depth, at = [""], 0, m.end()
        while depth >= 0:
            c = text[at]
            depth += (c in "([{") - (c in ")]}")
            if c == "," and depth == 0:
                args.append("")
            elif depth >= 0:
                args[-1] += c
            at += 1
        yield [a.strip() for a in args]


def test_range_checked_buffer_loads_have_no_scalar_offset():
    """A buffer load's range check is promised for the lane's offset alone: where a buffer's size keeps lanes out (rows
    past the end of a tile), the whole offset has to be the lane's."""
    seen = 0
    for name, text in _sources():
        sizes = [a[2] for a in _calls(text, "__builtin_amdgcn_make_buffer_rsrc")]
        loads = list(_calls(text, "__builtin_amdgcn_raw_ptr_buffer_load_lds"))
        if not loads or all(s == "0x7FFFFFFF" for s in sizes):  # nothing is kept out there: every address is inside
            continue
        for a in loads:
            assert a[4] == "0", (name, a)
            seen += 1
    assert seen
