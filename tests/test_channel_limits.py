"""Sizes that a launch does not take (2^32 threads or more) are refused on the CPU, before any HIP call.

No test here reaches a launch: the fake device addresses are never dereferenced."""
import pytest

from test_channel_abi import BF16, F32, UNSUPPORTED, T, bwd, fwd, gbwd, gfwd, norm, rec, scan, step, token


def at(place, shape, dtype, stride=None):
    """A tensor far from the others, in a range that fits it."""
    t = T(shape, dtype, 0, stride)
    t.data = 1 << 34 | place << 46
    return t


def wide_rec(B, L, C, dt):
    p = rec(B=1, L=20, C=4, dt=dt, flags=scan.SS_REC_LEAK)
    full, st = [B, L, C], [B, C]
    for n, (k, shape, d) in enumerate((
            ("x", full, dt), ("g", full, dt), ("i", full, dt), ("rate", [C], F32), ("si", st, F32), ("sf", st, F32),
            ("mk", [B, -(-L // 16), C], F32), ("h", full, dt), ("dh", full, dt), ("df", st, F32), ("dx", full, dt),
            ("dg", full, dt), ("di", full, dt), ("dr", [C], F32), ("d0", st, F32))):
        p[k] = at(n, shape, d)
    p["n"] = p["st"] = p["ws"] = None
    return p


# batch, L, channels, dtype, and which of forward and backward ask for 2^32 threads or more.  A forward block has a
# wave for each 16 tokens, 8 at most, a backward block one for each 8; 64 channels a wave, 128 in pairs of bf16
REC = [
    (1 << 20, 1024, 1, F32, True, True), (1 << 20, 1, 4096, F32, True, True), (1 << 20, 1, 4096, BF16, False, True),
    (1 << 20, 512, 64, F32, False, True), (1 << 20, 897, 2, BF16, True, True), (1 << 20, 896, 2, BF16, False, True),
    (1, (1 << 30) - 127, 1, F32, True, True), (1, (1 << 29) - 63, 64, BF16, False, True),
    (1 << 20, 1, 8192, BF16, True, True),
]


@pytest.mark.parametrize("B,L,C,dt,no_fwd,no_bwd", REC, ids=str)
def test_gatedrec_launches(B, L, C, dt, no_fwd, no_bwd):
    p = wide_rec(B, L, C, dt)
    ws = scan.lib().ss_gatedrec_workspace
    if no_fwd:
        assert ws(B, L, C, dt, 0) == UNSUPPORTED and fwd(p) == UNSUPPORTED
    else:
        assert ws(B, L, C, dt, 0) >= 0
    if no_bwd:
        assert ws(B, L, C, dt, 1) == UNSUPPORTED and bwd(p) == UNSUPPORTED
    else:
        assert ws(B, L, C, dt, 1) >= 0


def test_gatedrec_rows_of_single_channels():
    """bf16 rows that are not aligned to pairs take twice the blocks; the workspace's size does not tell."""
    p = wide_rec(1 << 20, 896, 128, BF16)
    for k in ("x", "g", "i", "dh"):
        p[k].data += 2
    assert scan.lib().ss_gatedrec_workspace(1 << 20, 896, 128, BF16, 0) >= 0
    assert fwd(p) == UNSUPPORTED and bwd(p) == UNSUPPORTED


@pytest.mark.parametrize("B,C,dt,shift", [(1 << 20, 4096, F32, 0), (1 << 20, 8192, BF16, 0), (1 << 20, 4096, BF16, 2),
                                          (1 << 20, 1 << 24, BF16, 0)])
def test_step_launches(B, C, dt, shift):
    p = token(flags=0)
    for n, k in enumerate(("x", "g", "i", "s", "so", "h")):
        p[k] = at(n, [B, C], F32 if k in ("s", "so") else dt)
    p["x"].data += shift
    p["rate"] = None
    assert step(p) == UNSUPPORTED


def wide_norm(B, L, C, G, xt, yt):
    p = norm()
    full = [B, L, C]
    for n, (k, shape, d) in enumerate((("x", full, xt), ("w", [C], F32), ("b", [C], F32), ("st", [B, G, 3], F32),
                                       ("y", full, yt), ("dy", full, yt), ("dx", full, xt), ("dw", [C], F32),
                                       ("db", [C], F32))):
        p[k] = at(n, shape, d)
    p.update(groups=G, n=None, ws=None)
    return p


# batch, L, channels, groups, x, y: a block of 256 threads for each row and group (resident or joined), 1024 for
# large resident groups, blocks of tiles by slabs of channels
NORM = [
    (1 << 20, 1, 128, 16, BF16, BF16), (1 << 20, 1, 16, 16, F32, F32), (1 << 20, 1, 64, 16, F32, F32),
    (1 << 20, 4, 96, 24, F32, F32), (1 << 20, 4, 96, 24, BF16, F32), (1 << 20, 40000, 8, 1, F32, BF16),
]


@pytest.mark.parametrize("B,L,C,G,xt,yt", NORM, ids=str)
def test_groupnorm_launches(B, L, C, G, xt, yt):
    p = wide_norm(B, L, C, G, xt, yt)
    assert gfwd(p) == UNSUPPORTED and gbwd(p) == UNSUPPORTED
    for back in (0, 1):
        assert scan.lib().ss_groupnorm_workspace(B, L, C, G, back) == UNSUPPORTED


def test_groupnorm_launches_by_form():
    """Sizes that some types and alignments take and others do not: the call decides."""
    p = wide_norm(1 << 20, 1000, 320, 4, BF16, BF16)      # 1024 threads a group; tiles of f32 are fewer
    assert scan.lib().ss_groupnorm_workspace(1 << 20, 1000, 320, 4, 0) >= 0 and gfwd(p) == UNSUPPORTED
    p = wide_norm(1 << 20, 256, 200, 1, BF16, BF16)
    for k in ("x", "y", "dy", "dx"):
        p[k].data += 2                                     # one channel an access: 25 slabs of 8
    assert gfwd(p) == UNSUPPORTED and gbwd(p) == UNSUPPORTED


def test_sizes_that_launch():
    """One below the limits: the workspace is given, as it was."""
    lib = scan.lib()
    for args in ((1 << 20, 512, 1), (1 << 20, 1, 4032), (1, 1 << 24, 64), (1, 1 << 20, 4096)):
        assert lib.ss_gatedrec_workspace(*args, F32, 0) >= 0, args
    for args in ((1 << 20, 4, 15 * 8, 15), (1 << 16, 1, 2048, 32), (1 << 20, 8, 4104, 1), (1, 1 << 24, 64, 2)):
        assert lib.ss_groupnorm_workspace(*args, 0) >= 0 and lib.ss_groupnorm_workspace(*args, 1) >= 0, args


def test_the_bounds_that_are_documented():
    """Sizes within the header's sufficient bounds are never refused."""
    lib = scan.lib()
    for e in range(21):
        for L in (1, 7, 64, 65, 100, 128, 129, 1000, 1 << 20, (1 << 28) - 9):
            for C in (1, 64, 65, 200, 4096, 1 << 20):
                B = 1 << e
                if B * -(-C // 64) * (L / 8 + 8) < 1 << 26:
                    for dt in (F32, BF16):
                        assert min(lib.ss_gatedrec_workspace(B, L, C, dt, back) for back in (0, 1)) >= 0, (B, L, C)
                for G in (1, 4, 32):
                    if C % G == 0 and B * G < 1 << 22 and B * -(-C // 8) * -(-L // 256) < 1 << 24:
                        assert min(lib.ss_groupnorm_workspace(B, L, C, G, back) for back in (0, 1)) >= 0, (B, L, C, G)
