"""The tile shapes the feed-forward products take, and the order of loads and
reads in their LDS rings, on the host.  Nothing here needs a GPU."""
import pytest

pytest.importorskip("torch")
from tests import ffn_shapes

bi = pytest.importorskip("deterministic_persistent_gemm_amd")

STREAM, ALL, TURNS = 0, 1, 2


def mx_shapes():
    """Every tile shape of the 4-bit product that some size takes."""
    seen = {}
    for dt in (bi.BI_BF16, bi.BI_F32):
        for M in (1, 4, 16, 17, 33, 64, 100, 130, 258, 400, 700, 1030, 2048, 4096):
            for N in (16, 272, 1024, 4096, 6288, 8720, 12288):
                for K in (32, 416, 1184, 4096):
                    t = bi.ffn_tile(bi.BI_FFN_MXFP4, M, N, K, dt)
                    seen[t["shape"]] = t
    return seen


def scale_events(t, stages):
    """What happens to a workgroup's scale ring, in the order in which nothing but
    the kernel's own waits and barriers holds it: ("write", group) when a load of
    a group may land, ("read", group) from when a wave may ask for it, ("got",
    group) once the value is known to be in every wave's registers."""
    kb, ring = t["stage_slices"], t["ring_stages"]
    parts = 4 // kb                                   # stages that bring a group after theirs
    brings = lambda st: st // parts + 1
    group = lambda s: s // 4
    ev = [("write", 0)] + [("write", brings(st)) for st in range(ring - 1)]
    if t["kernel"] == ALL:
        # slice s + 1 is read in step s; its values are known to have arrived when
        # its matrix instructions have been issued, in step s + 1; a stage's last step
        # starts with a barrier, after which a later stage's loads are issued
        ev.append(("read", 0))
        for s in range(stages * kb):
            if s % kb == kb - 1:
                ev.append(("write", brings(s // kb + ring - 1)))
            ev.append(("read", group(s + 1)))
            ev.append(("got", group(s)))
        return ev
    # in turns: reads are waited for at the barrier that ends a turn
    assert t["kernel"] == TURNS and kb == 2 and ring == 2
    first, second = [[] for _ in range(4 * stages + 4)], [[] for _ in range(4 * stages + 4)]
    for st in range(stages):
        for j in (0, 1):
            first[4 * st + 2 * j] += [("read", group(2 * st + j)), ("got", group(2 * st + j))]
            second[4 * st + 2 * j + 1] += [("read", group(2 * st + j)), ("got", group(2 * st + j))]
        first[4 * st].insert(0, ("write", brings(st + 1)))
        first[4 * st + 1].insert(0, ("write", brings(st + 1)))
        second[4 * st + 4].insert(0, ("write", brings(st + 2)))
    second[0].insert(0, ("write", brings(1)))
    # within a turn the two groups of waves run in any order: each one's reads are
    # open for the whole turn
    for a, b in zip(first, second):
        both = a + b
        ev += [e for e in both if e[0] == "read"] + [e for e in both if e[0] == "write"] + [e for e in both if e[0] == "got"]
    return ev


def overwritten(t, stages=40):
    """Scale groups that a load may overwrite while a read of them is open, or
    before their last read."""
    groups, faults, open_reads = t["scale_groups"], [], {}
    ev = scale_events(t, stages)
    last = {g: i for i, (what, g) in enumerate(ev) if what == "got"}
    for i, (what, g) in enumerate(ev):
        if what == "write":
            old = g - groups
            if old >= 0 and (open_reads.get(old, 0) > 0 or last.get(old, -1) > i):
                faults.append((i, old))
        elif what == "read":
            open_reads[g] = open_reads.get(g, 0) + 1
        else:
            open_reads[g] -= 1
    return faults


def test_scale_ring_holds_every_group_until_it_has_been_read():
    shapes = mx_shapes()
    assert sorted(shapes) == [0, 1, 2, 3, 4, 5]
    assert {t["kernel"] for t in shapes.values()} == {STREAM, ALL, TURNS}
    for t in shapes.values():
        if t["kernel"] == STREAM:
            # a stage brings its own groups, and its slot is refilled after the
            # barrier at which every wave waits for its reads of the stage
            assert t["stage_slices"] % 4 == 0 and t["scale_groups"] == t["ring_stages"] * t["stage_slices"] // 4
        else:
            assert overwritten(t) == [], t


def test_a_ring_one_group_too_small_is_found():
    """The model above sees the fault it is there for."""
    for t in mx_shapes().values():
        if t["kernel"] != STREAM:
            assert overwritten(dict(t, scale_groups=t["scale_groups"] - 1))


def test_refusals():
    out = (bi._I32 * 8)()
    tile = bi.lib().bi_lab_ffn_tile
    assert tile(9, 4, 32, 64, 1, out) == tile(1, 0, 32, 64, 1, out) == tile(1, 4, 32, 64, 7, out) == bi.BI_EINVAL
    assert tile(1, 4, 32, 64, 1, None) == bi.BI_EINVAL
    assert tile(1, 4, 24, 64, 1, out) == tile(1, 4, 32, 48, 1, out) == bi.BI_EUNSUPPORTED


def steady(op, sizes, dts):
    """Shapes that some size keeps busy for at least two stages past its ring, and
    two groups past its ring of scales."""
    seen = set()
    for M, N, K in sizes:
        for dt in dts:
            t = bi.ffn_tile(op, M, N, K, dt)
            k = {bi.BI_FFN_DX: N, bi.BI_FFN_DW: M}.get(op, K)
            slices = -(-k // t["slice_k"])
            if slices >= (t["ring_stages"] + 1) * t["stage_slices"] + 1 and (
                    not t["scale_groups"] or -(-slices // 4) >= t["scale_groups"] + 2):
                seen.add((t["shape"], dt))
    return seen


BF, F32 = bi.BI_BF16, bi.BI_F32


@pytest.mark.parametrize("op,sizes,shapes,dts", [
    (bi.BI_FFN_GATED, ffn_shapes.GATED, range(7), (BF,)), (bi.BI_FFN_MXFP4, ffn_shapes.MXFP4, range(6), (BF, F32)),
    (bi.BI_FFN_DX, ffn_shapes.LINEAR_BWD, range(7), (BF,)), (bi.BI_FFN_DW, ffn_shapes.LINEAR_BWD, range(1, 5), (BF, F32))],
    ids=["gated", "mxfp4", "dx", "dw"])
def test_every_shape_is_tested_past_its_ring(op, sizes, shapes, dts):
    seen = steady(op, sizes, (BF, F32) if op == bi.BI_FFN_DX else dts)
    for shape in shapes:
        for dt in dts:
            assert (shape, dt) in seen or (op == bi.BI_FFN_DX and (shape, F32) in seen), (shape, dt)
