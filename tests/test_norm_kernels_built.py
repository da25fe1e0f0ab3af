"""The norm's kernels in the library are those that a call reaches: for each direction one team (vectors
a thread, threads) a range of widths, in both types, with and without a ragged width, for every gate."""
import re


def test_only_reachable_teams():
    import ssm_sequence_models_amd as ssm
    with open(ssm.LIB_PATH, "rb") as f:
        names = set(re.findall(rb"norm_(fwd|bwd)_kernelINS_\d(BF16|F32)ELb([01])ELi(\d+)ELi(\d+)ELi([012])E", f.read()))
    teams = {b"fwd": {(1, 64), (2, 64), (1, 256), (2, 256), (1, 1024), (2, 1024)},
             b"bwd": {(1, 64), (2, 64), (1, 256), (1, 512), (1, 1024), (2, 1024)}}
    want = {(d, t, tail, b"%d" % nv, b"%d" % tpr, gate) for d in teams for nv, tpr in teams[d]
            for t in (b"BF16", b"F32") for tail in (b"0", b"1") for gate in (b"0", b"1", b"2")}
    assert names == want, sorted(names ^ want)
