"""The binding refuses what lies on another device than the current one, also
what it took in an earlier call (CPU only)."""
import pytest
import torch

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000   # never dereferenced


@pytest.fixture(scope="module")
def rq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_linear_layers_gb300 as rq
    return rq


class Weight:
    """As much of a dense f32 tensor on device 0 as the binding looks at."""

    dtype = torch.float32

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return 64

    def data_ptr(self):
        return A


def test_weights_of_norms_on_another_device(rq, monkeypatch):
    monkeypatch.setattr(rq._types, "device", lambda: 0, raising=False)
    params = [rq.NormParams(64, post_weight=Weight()), rq.NormParams(64, pre_weight=Weight())]
    plain = rq.NormParams(64)
    rows = dict(dtype=0, h_dtype=0, stream=0)
    for p in params + [plain]:
        rq.rq_residual_norm(p, B, C, D, 0x50000, 0, **rows)    # no tokens
    monkeypatch.setattr(rq._types, "device", lambda: 1)
    with pytest.raises(rq.RqError):
        rq.NormParams(64, post_weight=Weight())
    for p in params:
        with pytest.raises(rq.RqError) as e:
            rq.rq_residual_norm(p, B, C, D, 0x50000, 0, **rows)
        assert e.value.status == 2
    rq.rq_residual_norm(plain, B, C, D, 0x50000, 0, **rows)
