"""The gated recurrence on rows of whole pieces without masks (GPU), in every form and over many chunks and
hand-overs, against float64; and masked rows of the same sizes.  Tolerances as in test_gatedrec_gpu."""
import pytest

from gpu_helpers import say, torch_dev
from test_gatedrec_gpu import check, make, run, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mix", ["none", "leak", "unit"])
@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_form(mix, rate, gate, dtype):
    """Three chunks, the last of one piece; gates from shut to wide open."""
    torch = torch_dev()
    say("[rec] whole %s rate=%s gate=%s %s" % (mix, rate, gate, dtype))
    p = make(torch, 2, 272, 66, dtype, gate=gate, rate=rate, seed=4, spread=6.0)
    check(run(torch, p, mix, masks=False, states=True), want(p, mix, masks=False, states=True))


# L, C, dtype, gate, rate, mix, masks: more than 2048 tokens are more than one hand-over of the state
LONG = [
    (4096, 130, "bf16", True, True, "unit", False), (4096, 128, "bf16", False, False, "leak", False),
    (4112, 64, "bf16", True, False, "none", False), (4096, 65, "f32", True, True, "unit", False),
    (5000, 40, "f32", False, True, "leak", False), (3000, 31, "bf16", True, True, "unit", False),
    (4096, 130, "bf16", True, True, "unit", True), (4096, 66, "f32", False, False, "leak", True),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_rows(case):
    torch = torch_dev()
    L, C, dtype, gate, rate, mix, masks = case
    say("[rec] long %s" % (case,))
    # gates wide open: memories of up to 1000 tokens cross the hand-overs
    p = make(torch, 2, L, C, dtype, gate=gate, rate=rate, seed=L + C, spread=2.0)
    p["g"] = p["g"] + 3 if not rate else p["g"]
    p["starts"] = (torch.rand(2, L, generator=torch.Generator().manual_seed(L)) < 0.002).to(torch.int32).cuda()
    check(run(torch, p, mix, masks=masks, states=True), want(p, mix, masks=masks, states=True))


def test_masks_that_mask_nothing():
    """lengths of L and starts of zero: the same results up to rounding, by the other kernels."""
    torch = torch_dev()
    for dtype in ("f32", "bf16"):
        p = make(torch, 2, 640, 130, dtype, gate=True, rate=True, seed=6)
        p["lengths"][:] = 640
        p["starts"][:] = 0
        exp = want(p, "unit", masks=False, states=True)
        check(run(torch, p, "unit", masks=True, states=True), exp)
        check(run(torch, p, "unit", masks=False, states=True), exp)
