"""The sequence operators against their references by a comparison that no NaN passes, with memory that held NaN
before the calls: an output that is left unwritten, or that something behind a row's end has reached, shows."""
import pytest
import torch

from . import strict, test_gpu_distill, test_gpu_ln, test_gpu_scan

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def compare_strictly(monkeypatch):
    for module in (test_gpu_scan, test_gpu_ln, test_gpu_distill):
        monkeypatch.setattr(module, "within", strict.within)
    # what the allocator hands out next: NaN in every type, from both of its pools
    torch.cuda.empty_cache()
    pieces = [torch.full((1 << 19,), 255, dtype=torch.uint8, device="cuda") for _ in range(32)]
    pieces.append(torch.full((1 << 29,), 255, dtype=torch.uint8, device="cuda"))
    del pieces


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", test_gpu_scan.SIZES + [(140, 150, 260), (250, 33, 75), (30, 700, 70), (3, 700, 1030),
                                                        (2, 900, 778), (1, 9000, 70)], ids=str)
@pytest.mark.parametrize("options", ["everything", "padded"])
def test_scan(options, size, dtype):
    test_gpu_scan.both_ways(size, dtype, **test_gpu_scan.OPTIONS[options])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", test_gpu_scan.SIZES, ids=str)
def test_scan_packed(size, dtype):
    test_gpu_scan.both_ways(size, dtype, **test_gpu_scan.OPTIONS["packed"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", test_gpu_ln.SIZES, ids=str)
@pytest.mark.parametrize("rms", [False, True])
def test_norm(rms, size, dtype):
    test_gpu_ln.both_ways(size, dtype, rms, residual=True)
    test_gpu_ln.both_ways(size, dtype, rms, residual=False, gamma=test_gpu_ln.SIZES.index(size) % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(300_001, 16), (150_000, 7), (100_003, 130)], ids=str)
def test_norm_of_many_rows(size, dtype):
    test_gpu_ln.both_ways(size, dtype, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", test_gpu_distill.SIZES + [(40, 796, 152), (700, 11516, 64), (9, 23000, 33)], ids=str)
def test_loss(size, dtype):
    i = len(str(size))
    z, ids, q, w = test_gpu_distill.inputs(size, dtype, 0, ("f32", "bf16")[i % 2], (torch.int32, torch.int64)[i // 2 % 2])
    test_gpu_distill.all_ways(z, ids, q, None if i % 3 == 2 else w, (1.0, 2.0, 0.7, 4.0)[i % 4], dtype, f"{size} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [130, 4099, 60001])
def test_loss_of_rows_apart(V, dtype):
    test_gpu_distill.test_rows_apart_and_in_place(V, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 2000, 70001])
def test_loss_of_masked_logits(V, dtype):
    test_gpu_distill.test_masked_logits(1.0, V, dtype)
