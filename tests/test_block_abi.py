"""Entry points of linear attention, rotary positions and the norms on the CPU: every invalid call is
refused during host-side validation, before any HIP call, and sizes of workspaces are consistent.

No test here reaches a kernel launch: every call is refused, or describes an empty problem, so the
fake device addresses are never dereferenced.
"""
import ctypes
import os

import pytest

scan = pytest.importorskip("selective_state_space_88_amd.scan")

if not os.path.exists(scan.LIB_PATH):
    pytest.skip("libssscan.so not built", allow_module_level=True)

NULL, DTYPE, SHAPE, STRIDE, FLAGS, UNSUPPORTED, ALIAS, SCRATCH = -1, -2, -3, -4, -5, -6, -7, -10
F32, BF16, I32 = scan.SS_F32, scan.SS_BF16, scan.SS_I32
STEP = 1 << 28   # disjoint fake ranges


def T(shape, dtype, place, stride=None, offset=0):
    d = scan.SSTensor()
    d.data = STEP * (place + 1) + offset
    d.dtype = dtype
    d.ndim = len(shape)
    if stride is None:
        stride, acc = [], 1
        for n in reversed(shape):
            stride.insert(0, acc)
            acc *= n
    for i, (n, s) in enumerate(zip(shape, stride)):
        d.shape[i] = n
        d.stride[i] = s
    return d


def R(t):
    return None if t is None else ctypes.byref(t)


def lin(B=2, L=10, H=4, Hq=4, Hk=2, Hv=2, K=16, V=24, dt=BF16):
    return dict(q=T([B, L, Hq, K], dt, 0), k=T([B, L, Hk, K], dt, 1), v=T([B, L, Hv, V], dt, 2), g=T([H], F32, 3),
                n=T([B], I32, 4), si=T([B, H, K, V], F32, 5), sf=T([B, H, K, V], F32, 6), o=T([B, L, H, V], dt, 7),
                ws=T([1 << 22], F32, 8), do=T([B, L, H, V], dt, 9), df=T([B, H, K, V], F32, 10),
                dq=T([B, L, Hq, K], dt, 11), dk=T([B, L, Hk, K], dt, 12), dv=T([B, L, Hv, V], dt, 13),
                di=T([B, H, K, V], F32, 14))


def fwd(p):
    return scan.lib().ss_linattn_fwd(R(p["q"]), R(p["k"]), R(p["v"]), R(p["g"]), 0.5, R(p["n"]), R(p["si"]), R(p["sf"]),
                                     R(p["o"]), R(p["ws"]), None)


def bwd(p):
    return scan.lib().ss_linattn_bwd(*(R(p[x]) for x in ("q", "k", "v", "g")), 0.5,
                                     *(R(p[x]) for x in ("n", "si", "do", "df", "dq", "dk", "dv", "di", "ws")), None)


def set_field(t, **kw):
    for k, v in kw.items():
        if k in ("shape", "stride"):
            for i, x in enumerate(v):
                getattr(t, k)[i] = x
        else:
            setattr(t, k, v)


LIN_BAD = [
    ("q", None, NULL), ("k", None, NULL), ("v", None, NULL), ("g", None, NULL),
    ("k", dict(dtype=F32), DTYPE), ("v", dict(dtype=F32), DTYPE), ("g", dict(dtype=BF16), DTYPE),
    ("n", dict(dtype=F32), DTYPE), ("si", dict(dtype=BF16), DTYPE), ("q", dict(dtype=I32), DTYPE),
    ("q", dict(ndim=3), SHAPE), ("g", dict(ndim=2), SHAPE), ("k", dict(shape=[2, 9]), SHAPE),
    ("v", dict(shape=[1]), SHAPE), ("n", dict(shape=[3]), SHAPE), ("si", dict(shape=[2, 4, 16, 23]), SHAPE),
    ("k", dict(shape=[2, 10, 3]), SHAPE), ("g", dict(shape=[5]), SHAPE), ("q", dict(shape=[2, -1]), SHAPE),
    ("q", dict(stride=[640, 64, 16, 2]), STRIDE), ("q", dict(stride=[640, -64]), STRIDE),
    ("n", dict(stride=[2]), STRIDE),
]


@pytest.mark.parametrize("name,change,code", LIN_BAD, ids=str)
@pytest.mark.parametrize("call", [fwd, bwd], ids=["fwd", "bwd"])
def test_linattn_refusals(call, name, change, code):
    p = lin()
    if change is None:
        p[name] = None
    else:
        set_field(p[name], **change)
    assert call(p) == code


def test_linattn_outputs():
    for call, outs in ((fwd, ("o",)), (bwd, ("dq", "dk", "dv"))):
        for name in outs:
            p = lin()
            p[name] = None
            assert call(p) == NULL
            p = lin()
            p[name].dtype = F32
            assert call(p) == DTYPE
            p = lin()
            p[name].shape[1] = 11
            assert call(p) == SHAPE
            p = lin()
            p[name].stride[1] = 0        # its own elements overlap
            assert call(p) == STRIDE
    p = lin()
    p["do"] = None
    assert bwd(p) == NULL
    p = lin()
    p["do"].shape[3] = 20
    assert bwd(p) == SHAPE


def test_linattn_aliases():
    for out in ("o", "sf"):
        for other in ("q", "k", "v", "g", "n", "si", "o", "sf"):
            if other != out:
                p = lin()
                p[out].data = p[other].data
                assert fwd(p) == ALIAS, (out, other)
    for out in ("dq", "dk", "dv", "di"):
        for other in ("q", "k", "v", "g", "n", "si", "do", "df", "dq", "dk", "dv", "di"):
            if other != out:
                p = lin()
                p[out].data = p[other].data
                assert bwd(p) == ALIAS, (out, other)
    # a workspace over a tensor of the call, misaligned, of another type
    p = lin()
    p["ws"].data = p["k"].data
    assert fwd(p) == ALIAS and bwd(p) == ALIAS
    p = lin()
    p["ws"].data += 4
    assert fwd(p) == STRIDE
    p = lin()
    p["ws"].dtype = BF16
    assert fwd(p) == DTYPE


def test_slices_of_one_buffer_are_told_apart():
    """Gradients written into one fused row buffer share nothing; one feature further they do."""
    B, L = 2, 10
    widths = dict(dq=4 * 16, dk=2 * 16, dv=2 * 24)
    row = sum(widths.values())

    def fused(shift):
        p = lin()
        at = 0
        for name, heads, dim in (("dq", 4, 16), ("dk", 2, 16), ("dv", 2, 24)):
            p[name] = T([B, L, heads, dim], BF16, 11, stride=[L * row, row, dim, 1], offset=2 * at)
            at += widths[name]
        p["dk"].data -= 2 * shift
        return p

    # refused for something that is checked after the aliases, or before them
    p = fused(0)
    p["ws"].dtype = BF16
    assert bwd(p) == DTYPE
    assert bwd(fused(1)) == ALIAS


def test_linattn_sizes():
    f = scan.lib().ss_linattn_workspace
    for bad in ((-1, 8, 4, 4, 4, 4, 16, 16), (1, -8, 4, 4, 4, 4, 16, 16), (1, 8, 4, 3, 4, 4, 16, 16), (1, 8, 0, 1, 1, 1, 16, 16)):
        assert f(*bad, BF16, 0) == SHAPE
    for bad in ((1, 8, 4, 4, 4, 4, 0, 16), (1, 8, 4, 4, 4, 4, 16, 257), (1, 1 << 31, 1, 1, 1, 1, 16, 16),
                (1 << 20, 8, 2, 2, 2, 2, 16, 16)):
        assert f(*bad, BF16, 0) == UNSUPPORTED
    assert f(1, 8, 4, 4, 4, 4, 16, 16, I32, 0) == DTYPE
    assert f(2, 1, 4, 4, 4, 4, 16, 16, BF16, 0) == 0
    assert f(1, 65536, 4, 4, 4, 4, 64, 64, BF16, 0) > 0
    # shared heads add one f32 gradient per head, of the larger shared tensor: they are summed in turn
    own, shared = (f(1, 4096, 8, 8, h, h, 64, 64, BF16, 1) for h in (8, 2))
    assert shared - own == 4096 * 8 * 64
    p = lin(L=70000, H=4)
    p["ws"].shape[0] = 16
    assert fwd(p) == SCRATCH and bwd(p) == SCRATCH


def test_linattn_empty():
    p = lin(B=0)
    assert fwd(p) == 0 and bwd(p) == 0
    p = lin(L=0)
    p["sf"] = p["di"] = None
    assert fwd(p) == 0 and bwd(p) == 0


def step(p):
    return scan.lib().ss_linattn_step(*(R(p[x]) for x in ("q", "k", "v", "g")), 0.5, R(p["s"]), R(p["so"]), R(p["o"]),
                                      None)


def step_problem(B=2, H=4, K=16, V=24, dt=BF16):
    return dict(q=T([B, 4, K], dt, 0), k=T([B, 2, K], dt, 1), v=T([B, 2, V], dt, 2), g=T([H], F32, 3),
                s=T([B, H, K, V], F32, 4), so=T([B, H, K, V], F32, 5), o=T([B, H, V], dt, 6))


@pytest.mark.parametrize("name,change,code", [
    ("q", None, NULL), ("s", None, NULL), ("so", None, NULL), ("o", None, NULL), ("g", None, NULL),
    ("k", dict(dtype=F32), DTYPE), ("s", dict(dtype=BF16), DTYPE), ("so", dict(dtype=BF16), DTYPE),
    ("s", dict(shape=[2, 4, 15]), SHAPE), ("o", dict(shape=[2, 3]), SHAPE), ("k", dict(shape=[2, 3]), SHAPE),
    ("so", dict(stride=[0]), STRIDE), ("q", dict(shape=[2, 4, 300]), SHAPE),
], ids=str)
def test_step_refusals(name, change, code):
    p = step_problem()
    if change is None:
        p[name] = None
    else:
        set_field(p[name], **change)
    assert step(p) == code


def test_step_state_is_in_place_or_apart():
    p = step_problem()
    p["so"].data = p["s"].data + 4 * 16 * 24     # the next head's state
    assert step(p) == ALIAS
    p = step_problem()
    p["so"].data = p["s"].data                   # the same place, other rows
    p["so"].stride[0] *= 2
    assert step(p) == ALIAS
    p = step_problem()
    p["o"].data = p["s"].data
    assert step(p) == ALIAS
    p = step_problem(B=0)
    assert step(p) == 0


def rope_problem(dt=BF16):
    return dict(x=T([2, 5, 4, 16], dt, 0), x2=T([2, 5, 2, 16], dt, 1), pos=T([2, 5], I32, 2), f=T([8], F32, 3),
                out=T([2, 5, 4, 16], dt, 4), out2=T([2, 5, 2, 16], dt, 5), flags=0, pos0=0)


def rope(p):
    return scan.lib().ss_rope(R(p["x"]), R(p["x2"]), R(p["pos"]), p["pos0"], R(p["f"]), 1.0, p["flags"], R(p["out"]),
                              R(p["out2"]), None)


@pytest.mark.parametrize("name,change,code", [
    ("x", None, NULL), ("f", None, NULL), ("out", None, NULL), ("out2", None, NULL), ("x2", None, NULL),
    ("x2", dict(dtype=F32), DTYPE), ("out", dict(dtype=F32), DTYPE), ("pos", dict(dtype=F32), DTYPE),
    ("f", dict(dtype=BF16), DTYPE), ("x", dict(dtype=I32), DTYPE), ("f", dict(shape=[9]), SHAPE),
    ("pos", dict(shape=[2, 4]), SHAPE), ("x2", dict(shape=[1]), SHAPE), ("out", dict(shape=[2, 5, 3]), SHAPE),
    ("x", dict(stride=[320, 64, 16, 2]), STRIDE), ("out", dict(stride=[0]), STRIDE), ("pos", dict(stride=[-5]), STRIDE),
], ids=str)
def test_rope_refusals(name, change, code):
    p = rope_problem()
    if change is None:
        p[name] = None
    else:
        set_field(p[name], **change)
    assert rope(p) == code


def test_rope_flags_aliases_and_range():
    p = rope_problem()
    p["flags"] = 4
    assert rope(p) == FLAGS
    p = rope_problem()
    p["out"].data = p["x"].data + 2              # shifted by a feature: not in place
    assert rope(p) == ALIAS
    p = rope_problem()
    p["out2"].data = p["x"].data
    assert rope(p) == ALIAS
    p = rope_problem()
    p["out"].data = p["f"].data
    assert rope(p) == ALIAS
    p = rope_problem()
    p["pos"], p["pos0"] = None, 1 << 60
    assert rope(p) == UNSUPPORTED


def add_problem(B=2, L=5, C=16):
    s = [B, L, C]
    return dict(x=T(s, BF16, 0), r=T(s, F32, 1), w=T([C], F32, 2), sum=T(s, F32, 3), y=T(s, BF16, 4), dy=T(s, BF16, 5),
                ds=T(s, F32, 6), dr=T(s, F32, 7), dx=T(s, BF16, 8), dw=T([C], F32, 9), ws=T([1 << 20], F32, 10), eps=1e-5)


def add_fwd(p):
    return scan.lib().ss_addnorm_fwd(R(p["x"]), R(p["r"]), R(p["w"]), 1.0, p["eps"], R(p["sum"]), R(p["y"]), None)


def add_bwd(p):
    return scan.lib().ss_addnorm_bwd(R(p["dy"]), R(p["ds"]), R(p["sum"]), R(p["w"]), 1.0, p["eps"], R(p["dr"]), R(p["dx"]),
                                     R(p["dw"]), R(p["ws"]), None)


@pytest.mark.parametrize("call,name,change,code", [
    (add_fwd, "x", None, NULL), (add_fwd, "w", None, NULL), (add_fwd, "y", None, NULL),
    (add_fwd, "r", dict(dtype=BF16), DTYPE), (add_fwd, "w", dict(dtype=BF16), DTYPE), (add_fwd, "y", dict(dtype=I32), DTYPE),
    (add_fwd, "r", dict(shape=[2, 4]), SHAPE), (add_fwd, "w", dict(shape=[15]), SHAPE), (add_fwd, "x", dict(ndim=2), SHAPE),
    (add_fwd, "x", dict(stride=[80, 1, 5]), STRIDE), (add_fwd, "y", dict(stride=[80, 8]), STRIDE),
    (add_bwd, "dy", None, NULL), (add_bwd, "sum", None, NULL), (add_bwd, "w", None, NULL),
    (add_bwd, "ds", dict(dtype=BF16), DTYPE), (add_bwd, "dr", dict(dtype=BF16), DTYPE), (add_bwd, "dw", dict(dtype=BF16), DTYPE),
    (add_bwd, "dy", dict(shape=[2, 4]), SHAPE), (add_bwd, "dw", dict(shape=[17]), SHAPE), (add_bwd, "dx", dict(stride=[0]), STRIDE),
], ids=str)
def test_addnorm_refusals(call, name, change, code):
    p = add_problem()
    if change is None:
        p[name] = None
    else:
        set_field(p[name], **change)
    assert call(p) == code


def test_addnorm_aliases_and_sizes():
    for call, pairs in ((add_fwd, (("y", "x"), ("y", "sum"), ("y", "r"), ("sum", "x"), ("sum", "w"))),
                        (add_bwd, (("dx", "dy"), ("dx", "ds"), ("dx", "dr"), ("dr", "sum"), ("dw", "w"), ("ws", "dy")))):
        for a, b in pairs:
            p = add_problem()
            p[a].data = p[b].data
            assert call(p) == ALIAS, (a, b)
    p = add_problem()
    p["sum"].data = p["r"].data + 64             # over the residual, but not the residual
    assert add_fwd(p) == ALIAS
    for eps in (-1e-6, float("nan")):
        p = add_problem()
        p["eps"] = eps
        assert add_fwd(p) == UNSUPPORTED and add_bwd(p) == UNSUPPORTED
    assert add_fwd(add_problem(C=32769)) == UNSUPPORTED
    p = add_problem()
    p["ws"].shape[0] = 3
    assert add_bwd(p) == SCRATCH
    assert add_fwd(add_problem(L=0)) == 0
    p = add_problem(L=0)
    p["dw"] = None
    assert add_bwd(p) == 0
    p = add_problem()
    p["dr"] = p["dx"] = p["dw"] = None           # nothing asked for
    assert add_bwd(p) == 0


def gate_problem(B=2, L=6, C=32):
    s = [B, L, C]
    return dict(x=T(s, BF16, 0), z=T(s, F32, 1), w=T([C], F32, 2), y=T(s, BF16, 3), dy=T(s, F32, 4), dx=T(s, BF16, 5),
                dz=T(s, F32, 6), dw=T([C], F32, 7), ws=T([1 << 20], F32, 8), groups=4, flags=0, eps=1e-5)


def gate_fwd(p):
    return scan.lib().ss_gatenorm_fwd(R(p["x"]), R(p["z"]), R(p["w"]), p["groups"], p["eps"], p["flags"], R(p["y"]), None)


def gate_bwd(p):
    return scan.lib().ss_gatenorm_bwd(R(p["dy"]), R(p["x"]), R(p["z"]), R(p["w"]), p["groups"], p["eps"], p["flags"],
                                      R(p["dx"]), R(p["dz"]), R(p["dw"]), R(p["ws"]), None)


@pytest.mark.parametrize("call,name,change,code", [
    (gate_fwd, "x", None, NULL), (gate_fwd, "w", None, NULL), (gate_fwd, "y", None, NULL),
    (gate_fwd, "z", dict(shape=[2, 5]), SHAPE), (gate_fwd, "w", dict(shape=[31]), SHAPE), (gate_fwd, "x", dict(dtype=I32), DTYPE),
    (gate_fwd, "x", dict(stride=[400, 64, 2]), STRIDE), (gate_fwd, "y", dict(stride=[0]), STRIDE),
    (gate_bwd, "dx", None, NULL), (gate_bwd, "dz", None, NULL), (gate_bwd, "z", None, NULL), (gate_bwd, "dy", None, NULL),
    (gate_bwd, "dx", dict(dtype=F32), DTYPE), (gate_bwd, "dz", dict(dtype=BF16), DTYPE), (gate_bwd, "dw", dict(shape=[4]), SHAPE),
    (gate_bwd, "dx", dict(stride=[192, 0]), STRIDE),
], ids=str)
def test_gatenorm_refusals(call, name, change, code):
    p = gate_problem()
    if change is None:
        p[name] = None
    else:
        set_field(p[name], **change)
    assert call(p) == code


def test_gatenorm_groups_flags_aliases():
    for groups, code in ((0, SHAPE), (-1, SHAPE), (5, SHAPE)):
        p = gate_problem()
        p["groups"] = groups
        assert gate_fwd(p) == code and gate_bwd(p) == code
    p = gate_problem()
    p["flags"] = 2
    assert gate_fwd(p) == FLAGS
    p = gate_problem()
    p["y"].data = p["x"].data
    assert gate_fwd(p) == ALIAS
    for a, b in (("dx", "x"), ("dz", "z"), ("dx", "dz"), ("dw", "w"), ("ws", "dx")):
        p = gate_problem()
        p[a].data = p[b].data
        assert gate_bwd(p) == ALIAS, (a, b)
    p = gate_problem()
    p["eps"] = float("nan")
    assert gate_fwd(p) == UNSUPPORTED
    p = gate_problem(C=4 * 32776)
    assert gate_fwd(p) == UNSUPPORTED
    p = gate_problem()
    p["ws"].shape[0] = 3
    assert gate_bwd(p) == SCRATCH
    assert gate_fwd(gate_problem(B=0)) == 0
    f = scan.lib().ss_norm_workspace
    assert f(2, 8, 30, 4) == SHAPE and f(1, 8, 40000, 1) == UNSUPPORTED and f(0, 8, 64, 1) == 0 and f(4, 8, 64, 2) > 0


def test_binding_refuses_cpu_tensors_and_other_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):
        scan.rope(x, torch.zeros(4))
    with pytest.raises(ValueError):
        scan.linattn_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError):
        scan.addnorm_fwd(x[0], torch.ones(8))


def test_rope_inv_freq_on_the_host():
    plain, amp = scan.rope_inv_freq(16, 10000.0)
    assert plain.shape == (16,) and amp == 1.0 and float(plain[0]) == 1.0
    assert scan.rope_inv_freq(0)[0].numel() == 0
    for kw in (dict(n=-1), dict(n=4, base=0.0), dict(n=4, factor=0.5), dict(n=4, scaling="no")):
        with pytest.raises(ValueError):
            scan.rope_inv_freq(**kw)


@pytest.mark.parametrize("call,problem,first,second", [
    (fwd, "lin", "o", "q"), (fwd, "lin", "o", "v"), (fwd, "lin", "sf", "si"), (bwd, "lin", "dq", "q"),
    (bwd, "lin", "dk", "dq"), (bwd, "lin", "dv", "do"), (bwd, "lin", "di", "df"), (step, "step", "o", "q"),
    (rope, "rope", "out", "x2"), (rope, "rope", "out", "out2"), (add_fwd, "add", "y", "r"), (add_fwd, "add", "sum", "x"),
    (add_fwd, "add", "sum", "y"), (add_bwd, "add", "dr", "sum"), (add_bwd, "add", "dx", "dr"), (add_bwd, "add", "dw", "w"),
    (gate_fwd, "gate", "y", "x"), (gate_fwd, "gate", "y", "z"), (gate_bwd, "gate", "dx", "x"),
    (gate_bwd, "gate", "dz", "dx"), (gate_bwd, "gate", "dw", "w")])
def test_one_descriptor_in_two_places(call, problem, first, second):
    """A caller may pass the same ss_tensor as two arguments: two views of one tensor all the same."""
    p = {"lin": lambda: lin(Hk=4, Hv=4, V=16, dt=F32), "step": lambda: step_problem(V=16),
         "rope": rope_problem, "add": add_problem, "gate": gate_problem}[problem]()
    if problem == "rope":
        p["x2"], p["out2"] = T([2, 5, 4, 16], BF16, 1), T([2, 5, 4, 16], BF16, 5)
    for t in p.values():
        if problem in ("add", "gate") and isinstance(t, scan.SSTensor):
            t.dtype = F32
    p[first] = p[second]
    assert call(p) == ALIAS


def test_rope_and_states_in_place_by_one_descriptor():
    """The in-place forms through one descriptor pass the checks (empty problems: nothing is launched)."""
    p = rope_problem()
    p["x"] = p["out"] = T([2, 0, 4, 16], BF16, 0)
    p["x2"] = p["out2"] = T([2, 0, 2, 16], BF16, 1)
    p["pos"] = T([2, 0], I32, 2)
    assert rope(p) == 0
    p = add_problem(L=0)
    p["sum"] = p["r"]
    assert add_fwd(p) == 0


def test_limits_of_launches():
    ws = scan.lib().ss_norm_workspace
    assert ws(1, 0, 1 << 24, 512) == 0 and ws(1, 0, (1 << 24) + 512, 512 + 1) == SHAPE
    assert ws(1, 0, 1 << 25, 1024) == UNSUPPORTED and ws(1, 0, 65536, 65536) == UNSUPPORTED
    assert ws(1 << 16, 1 << 15, 16, 1) == UNSUPPORTED and ws(1 << 15, 1 << 15, 16, 1) > 0
    p = gate_problem(C=1 << 25)
    p["groups"] = 1024
    assert gate_fwd(p) == UNSUPPORTED and gate_bwd(p) == UNSUPPORTED
    lw = scan.lib().ss_linattn_workspace
    assert lw(1 << 19, 1, 4, 4, 4, 4, 64, 64, BF16, 0) == UNSUPPORTED and lw(1, 1 << 31, 1, 1, 1, 1, 64, 64, F32, 1) == UNSUPPORTED
