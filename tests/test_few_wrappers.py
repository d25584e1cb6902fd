"""The few-token wrappers' host side, without a GPU: tensors that pass for a GPU's, launches that are recorded."""
import threading
import time

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


class SlowLibrary:
    """Sizes from the library; a launch takes a while, and notes whether another is under way on its workspace."""

    def __init__(self, lib):
        self.lib, self.busy, self.calls, self.shared = lib, set(), 0, 0

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)

        def launch(*args):
            ws = args[-3]
            self.calls += 1
            self.shared += ws in self.busy
            self.busy.add(ws)
            time.sleep(0.002)    # ctypes lets other threads run during a call
            self.busy.discard(ws)
            return 0
        return launch


@pytest.fixture
def one_stream(monkeypatch, lib):  # noqa: F811
    """All threads on one stream of one device, workspaces in host memory."""
    slow = SlowLibrary(lib)
    monkeypatch.setattr(few, "load", lambda: slow)
    monkeypatch.setattr(few, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(few, "_current_device", lambda: 0)
    monkeypatch.setattr(few, "_is_capturing", lambda: False)
    monkeypatch.setattr(few, "alloc_workspace", lambda n, device: torch.zeros(n, dtype=U8))
    monkeypatch.setattr(few, "_scratch_cache", {})
    return slow


def test_calls_of_two_threads_do_not_mix_on_one_workspace(one_stream):
    x, out = on_gpu(20, 256, dtype=BF16), on_gpu(20, 40, dtype=BF16)
    codes, scales = on_gpu(40, 128, dtype=U8), on_gpu(40, 8, dtype=BF16)
    idx, gates = on_gpu(20, 2, dtype=I32), on_gpu(20, 2, dtype=F32)
    w13, w2, y = on_gpu(3, 16, 256, dtype=BF16), on_gpu(3, 256, 8, dtype=BF16), on_gpu(20, 256, dtype=BF16)

    def work():
        for _ in range(10):
            few.w4_linear(x, codes, scales, out=out)
            few.moe_swiglu(x, idx, gates, w13, w2, out=y)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert one_stream.calls == 80 and one_stream.shared == 0


def test_a_large_workspace_is_not_kept(one_stream):
    codes, scales = on_gpu(8, 16, dtype=U8), on_gpu(8, 1, dtype=BF16)
    sizes = []
    for rows in (1, 30000, 20, 400000, 1):    # scratch of 0, 10, 0.1 and 133 MB
        few.w4_linear(on_gpu(rows, 32, dtype=BF16), codes, scales, out=on_gpu(rows, 8, dtype=BF16))
        sizes.append(sum(ws.numel() for ws in few._scratch_cache.values()))
    assert sizes[0] < 1 << 20 < 8 << 20 < sizes[1] == sizes[-1] <= few._KEEP_BYTES
    assert one_stream.calls == 5


def test_moe_layer_refuses_to_drop_gradients(launches, monkeypatch):
    monkeypatch.setattr(few, "moe_route", lambda *args: ("idx", "gates"))
    monkeypatch.setattr(few, "moe_swiglu", lambda *args, workspace: "bf16")
    monkeypatch.setattr(few, "moe_swiglu_w4", lambda *args, workspace: "4 bits")
    plain = [on_gpu(*s, dtype=BF16) for s in ((2, 64), (3, 64), (3, 16, 64), (3, 64, 8))]
    q13, q2 = ((on_gpu(3, n, K // 2, dtype=U8), on_gpu(3, n, 1, dtype=BF16), None) for n, K in ((16, 64), (64, 8)))
    assert few.moe_layer(*plain, 1) == "bf16" and few.moe_layer(*plain[:2], q13, q2, 1) == "4 bits"
    for i in range(4):
        args = list(plain)
        args[i] = torch.zeros(plain[i].shape, dtype=BF16, requires_grad=True)
        with pytest.raises(RuntimeError, match="no_grad"):
            few.moe_layer(*args, 1)
        if i < 2:
            with pytest.raises(RuntimeError, match="no_grad"):
                few.moe_layer(*args[:2], q13, q2, 1)
        with torch.no_grad():
            assert few.moe_layer(*args, 1) == "bf16"
    scales = torch.zeros(q2[1].shape, dtype=BF16, requires_grad=True)
    with pytest.raises(RuntimeError, match="no_grad"):
        few.moe_layer(*plain[:2], q13, (q2[0], scales, None), 1)
