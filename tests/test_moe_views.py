"""Views whose rows overlap (expanded, or with a pitch below their width): the
routing and FP8B128 entry points get the pitch that the tensor has, and refuse
it on the host.  Host tensors stand in for the GPU's: no call gets past the refusal."""
import pytest
import torch


@pytest.fixture
def refused(monkeypatch):
    import block_scaled_precision_bsq_amd as bsq
    monkeypatch.setattr(bsq, "_dev", lambda t, name, dtypes: t)
    monkeypatch.setattr(bsq, "_stream", lambda stream=None: None)

    def check(name, at, pitch, call):
        """The call passes `pitch` as argument `at` of entry point `name`, which refuses it."""
        real = getattr(bsq._lib, name)

        def entry(*args):
            assert args[at] == pitch
            return real(*args)

        monkeypatch.setattr(bsq._lib, name, entry)
        with pytest.raises(bsq.BsqError) as e:
            call(bsq)
        assert e.value.status == bsq.BSQ_ERR_INVALID_ARG
        monkeypatch.setattr(bsq._lib, name, real)

    return check


def views(rows, cols, dtype):
    """(view, pitch): one row for all, one value for all, rows that overlap by half."""
    yield torch.zeros(1, cols, dtype=dtype).expand(rows, cols), 0
    yield torch.zeros(rows * cols, dtype=dtype).as_strided((rows, cols), (cols // 2, 1)), cols // 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(refused, dtype):
    T, E, K = 6, 16, 2
    ids, w, lse = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T)
    counts = torch.zeros(E + 1, dtype=torch.int32)
    for l, pitch in views(T, E, dtype):
        refused("bsq_moe_route", 4, pitch, lambda b: b.bsq_moe_route(l, K))
        refused("bsq_moe_route_bwd", 4, pitch, lambda b: b.bsq_moe_route_bwd(l, ids, w, lse, counts))
        refused("bsq_moe_route_bwd", 16, pitch,
                lambda b: b.bsq_moe_route_bwd(torch.zeros(T, E, dtype=dtype), ids, w, lse, counts, dlogits=l))


def test_quantize(refused):
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    idx = torch.zeros(9, dtype=torch.int32)
    for x, pitch in views(6, 32, torch.bfloat16):
        refused("bsq_quantize_fp8b128", 3, pitch, lambda b: b.bsq_quantize_fp8b128(x))
        refused("bsq_quantize_fp8b128", 3, pitch, lambda b: b.bsq_quantize_fp8b128(x, offsets=off))
        refused("bsq_quantize_fp8b128", 3, pitch, lambda b: b.bsq_quantize_fp8b128(x, row_index=idx))
        refused("bsq_quantize_fp8b128_weights", 4, pitch, lambda b: b.bsq_quantize_fp8b128_weights(x, 2))


def test_combine(refused):
    slot = torch.zeros(6, 2, dtype=torch.int32)
    full = torch.zeros(6, 32)
    for x, pitch in views(6, 32, torch.float32):
        refused("bsq_moe_combine", 4, pitch, lambda b: b.bsq_moe_combine(x, slot))
        refused("bsq_moe_combine", 10, pitch, lambda b: b.bsq_moe_combine(full, slot, y=x))
        refused("bsq_moe_combine_bwd", 4, pitch, lambda b: b.bsq_moe_combine_bwd(x, full, slot))
        refused("bsq_moe_combine_bwd", 7, pitch, lambda b: b.bsq_moe_combine_bwd(full, x, slot))
        refused("bsq_moe_combine_bwd", 14, pitch, lambda b: b.bsq_moe_combine_bwd(full, full, slot, dye=x))
