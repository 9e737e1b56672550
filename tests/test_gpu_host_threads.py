"""The C entry points from several host threads at once (ctypes lets go of the interpreter's lock), each on a stream of
its own, with launches of differing shared memory: every result is the one that a single thread gets."""
import threading

import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

pytestmark = pytest.mark.gpu


def loss_call(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((6, V), device="cuda", generator=g)
    ids = torch.randint(0, V, (6, 20), device="cuda", generator=g, dtype=torch.int32)
    q, loss, dz = torch.randn((6, 20), device="cuda", generator=g), torch.empty(6, device="cuda"), torch.empty_like(z)
    d = train.make_distill_desc(z, ids, q, 1.5)

    def call(stream):
        train.conv_distill_grad(d, z, ids, q, None, 0.5, loss, dz, stream)
    return call, (loss, dz)


def norm_call(D):
    g = torch.Generator(device="cuda").manual_seed(D)
    x, dy = (torch.randn((300, D), device="cuda", generator=g) for _ in range(2))
    _, _, mean, rstd = train.layer_norm(x)
    d = train.make_ln_desc(300, D, torch.float32)
    ws = torch.empty(train.conv_ln_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")

    def call(stream):
        train.conv_ln_bwd(d, x, dy, None, mean, rstd, None, dx, dg, db, ws, stream)
    return call, (dx, dg, db)


def test_four_threads():
    work = [[loss_call(V) for V in (3000 + 901 * k, 100000 + 7 * k, 40000 - 333 * k, 12000)]
            + [norm_call(D) for D in (200 + k, 1430, 4000 + 8 * k)] for k in range(4)]
    torch.cuda.synchronize()
    failed, gate = [], threading.Barrier(len(work))
    streams = [torch.cuda.Stream() for _ in work]

    def run(calls, stream):
        try:
            gate.wait(30)
            for _ in range(20):
                for call, _ in calls:
                    call(stream)
        except Exception as e:  # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=run, args=a) for a in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for calls in work:
        for call, outputs in calls:
            got = [t.clone() for t in outputs]
            for t in outputs:
                t.fill_(float("nan"))
            call(None)
            assert all(torch.equal(a, b) for a, b in zip(got, outputs))
    assert train.binding.conv_device_status() == 0
