"""The group norm's backward without the forward's ``stats``, on the CPU: refused before any HIP call.

No test here reaches a launch: the fake device addresses are never dereferenced."""
import pytest

from test_channel_abi import BF16, F32, NULL, gbwd, norm


@pytest.mark.parametrize("C,G,t", [(24, 3, BF16), (24, 4, BF16), (16, 4, F32)])
@pytest.mark.parametrize("L", [0, 20])
def test_groupnorm_backward_needs_stats(C, G, t, L):
    """``stats`` of rows that are there, without data, whether or not the rows have positions."""
    for drop in ((), ("dw",), ("db",)):
        p = norm(L=L, C=C, G=G, xt=t, yt=t)
        for k in drop:
            p[k] = None
        p["st"].data = None
        p["n"] = None
        assert gbwd(p) == NULL, drop
