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


def _body(text, name):
    """The body of the function `name`."""
    at = text.index("{", text.index(name + "("))
    depth, end = 1, at + 1
    while depth:
        depth += (text[end] == "{") - (text[end] == "}")
        end += 1
    return text[at:end]


def test_lanes_that_share_lds_are_ordered():
    """Where lanes of one wave write, add to and read each other's places in LDS, a fence of the wave stands between:
    each lane's own accesses alone would let the compiler move or forward them."""
    text = dict(_sources())["moe_balance.hip"]
    sync = r"wave_sync\(\);"
    assert re.search(r"__builtin_amdgcn_fence\(__ATOMIC_RELEASE, \"wavefront\"\);\s*__builtin_amdgcn_wave_barrier\(\);\s*"
                     r"__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, \"wavefront\"\);", _body(text, "void wave_sync"))
    for kernel, steps in (("route_backward_kernel", (r"rows\[[^;]*\] = v\[", r"atomicAdd\(&rows\[", r"= rows\[")),
                          ("balance_small_kernel", (r"count\[[^;]*\] = 0;", r"add_picks\([^;]*count"))):
        body = _body(text, kernel)
        at = [[m.start() for m in re.finditer(s, body)] for s in steps]
        assert all(len(a) == 1 for a in at), (kernel, at)
        for (a,), (b,) in zip(at, at[1:]):
            assert a < b and len(re.findall(sync, body[a:b])) == 1, (kernel, a, b)


def test_traffic_records_follow_every_source_of_the_layer(tmp_path, monkeypatch):
    """The hash that the layer's traffic records carry leaves out other operators' files by their whole names: a new
    source counts, whatever its name begins with."""
    import bench

    before = bench.kernel_source_hash()
    for path in glob.glob(os.path.join(CSRC, "*")):
        (tmp_path / os.path.basename(path)).write_bytes(open(path, "rb").read())
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    assert bench.kernel_source_hash() == before
    (tmp_path / "moe_fp8_tile.hip").write_text("// another")
    assert bench.kernel_source_hash() == before
    (tmp_path / "moe_fp8_layer.h").write_text("// new")
    assert bench.kernel_source_hash() != before
