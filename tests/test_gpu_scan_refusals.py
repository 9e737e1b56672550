"""The gated scan refuses companions that do not fit x, one at a time, before anything is enqueued: another size,
type, layout or machine; a good call with the same others goes through."""
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

pytestmark = pytest.mark.gpu
B, T, D = 3, 20, 8


def made(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def arguments():
    return dict(x=made(B, T, D), gate=made(B, T, D), h=made(B, T, D), dh=made(B, T, D), h0=made(B, D), dlast=made(B, D),
                reset=made(B, T, dtype=torch.bool), lengths=torch.full((B,), T, dtype=torch.int32, device="cuda"),
                out=made(B, T, D), last=made(B, D), dx=made(B, T, D), dgate=made(B, T, D))


FORWARD = ("x", "gate", "h0", "reset", "lengths", "out", "last")
BACKWARD = ("x", "gate", "h", "dh", "h0", "dlast", "reset", "lengths", "dx", "dgate")
STEPS = {  # (batch, time, channels)
    "sizes": lambda: made(B, T, D + 1), "steps": lambda: made(B, T - 1, D), "rows": lambda: made(B + 1, T, D),
    "dimensions": lambda: made(B * T, D), "type": lambda: made(B, T, D, dtype=torch.bfloat16),
    "double": lambda: made(B, T, D, dtype=torch.float64), "host": lambda: torch.zeros(B, T, D),
    "channels apart": lambda: made(B, D, T).transpose(1, 2), "expanded channels": lambda: made(B, T, 1).expand(B, T, D)}
STATES = {  # (batch, channels), fp32
    "sizes": lambda: made(B, D + 1), "rows": lambda: made(B + 1, D), "dimensions": lambda: made(B, 1, D),
    "type": lambda: made(B, D, dtype=torch.bfloat16), "host": lambda: torch.zeros(B, D),
    "strided": lambda: made(D, B).t()}
FLAGS = {
    "sizes": lambda: made(B, T + 1, dtype=torch.bool), "rows": lambda: made(B + 1, T, dtype=torch.bool),
    "dimensions": lambda: made(B, T, 1, dtype=torch.bool), "int32": lambda: made(B, T, dtype=torch.int32),
    "float": lambda: made(B, T), "host": lambda: torch.zeros(B, T, dtype=torch.bool),
    "strided": lambda: made(T, B, dtype=torch.bool).t()}
LENGTHS = {
    "sizes": lambda: made(B + 1, dtype=torch.int32), "dimensions": lambda: made(B, 1, dtype=torch.int32),
    "int64": lambda: made(B, dtype=torch.int64), "float": lambda: made(B), "host": lambda: torch.zeros(B, dtype=torch.int32),
    "strided": lambda: made(2 * B, dtype=torch.int32)[::2]}
KINDS = {"h0": STATES, "dlast": STATES, "last": STATES, "reset": FLAGS, "lengths": LENGTHS}


def call(function, names, **other):
    a = {k: v for k, v in arguments().items() if k in names}
    a.update(other)
    return function(**a)


@pytest.mark.parametrize("function,names", [(train.gated_scan, FORWARD), (train.gated_scan_bwd, BACKWARD)],
                         ids=["forward", "backward"])
def test_one_wrong_companion(function, names):
    call(function, names)
    for name in names:
        for what, make in KINDS.get(name, STEPS).items():
            with pytest.raises(ValueError):
                call(function, names, **{name: make()})
                pytest.fail(f"{name}: {what}")
        with pytest.raises(ValueError):
            call(function, names, **{name: 1.0})
    for name in ("x", "gate") + (("h", "dh") if "dh" in names else ()):
        with pytest.raises(ValueError):
            call(function, names, **{name: None})
    call(function, names)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["out", "dx", "dgate"])
def test_outputs_whose_rows_overlap(name):
    function, names = (train.gated_scan, FORWARD) if name == "out" else (train.gated_scan_bwd, BACKWARD)
    for t in (made(1, T, D).expand(B, T, D), made(B, 1, D).expand(B, T, D),
              torch.as_strided(made(B * T * D), (B, T, D), (T * D, D - 1, 1))):
        with pytest.raises(train.binding.ConvError):
            call(function, names, **{name: t})


def test_flags_of_both_types_and_views_go_through():
    a = arguments()
    want = train.gated_scan(a["x"], a["gate"], reset=a["reset"])
    got = train.gated_scan(a["x"], a["gate"], reset=a["reset"].view(torch.uint8))
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    wide = made(B, T, 2 * D)
    train.gated_scan(wide[..., :D], wide[..., D:], out=made(T, B, D).transpose(0, 1))
    expanded = made(1, 1, D).expand(B, T, D)   # an input's rows may be one
    train.gated_scan(expanded, a["gate"])
