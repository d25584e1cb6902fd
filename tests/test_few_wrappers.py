"""The few-token wrappers' host side, without a GPU: tensors that pass for a GPU's, launches that are recorded."""
import pytest
import torch

from expert_gemm_layers_gb300 import few
from test_few_refusals import lib  # noqa: F401  (fixture: builds the library)

BF16, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class OnGpu(torch.Tensor):
    """A host tensor that says it is on CUDA device 0."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def on_gpu(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def launches(monkeypatch, lib):  # noqa: F811
    """Launches are recorded as (function, arguments) instead of made."""
    made = []
    monkeypatch.setattr(few, "_launch", lambda fn, index, *args: made.append((fn, args)))
    return made


def test_w4_linear_checks_the_workspace_it_is_given(launches, lib):  # noqa: F811
    x, codes, scales = on_gpu(20, 256, dtype=BF16), on_gpu(40, 128, dtype=U8), on_gpu(40, 8, dtype=BF16)
    need, out = lib.dg_w4_linear_workspace_bytes(20, 256, 40), on_gpu(20, 40, dtype=BF16)
    for ws, error, match in ((torch.zeros(need, dtype=U8), ValueError, "CUDA"),          # a host address
                             (on_gpu(need, dtype=torch.int8), TypeError, "uint8"),
                             (on_gpu(2 * need, dtype=U8)[::2], ValueError, "contiguous"),
                             (on_gpu(need - 1, dtype=U8), ValueError, "needs"),
                             (need, TypeError, "tensor")):
        with pytest.raises(error, match=match):
            few.w4_linear(x, codes, scales, out=out, ws=ws)
    assert not launches
    ws = on_gpu(need, dtype=U8)
    few.w4_linear(x, codes, scales, out=out, ws=ws)
    assert len(launches) == 1 and launches[0][1][-2:] == (ws.data_ptr(), need)
