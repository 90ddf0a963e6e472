"""The torch side of the layer operators without a GPU: what a call hands to
the library, and what it refuses before that.  The library is replaced by a
record of its calls and tensors by stand-ins, so nothing is launched."""
import pytest
import torch

from mhc_hyper_connection_gb300 import build as mbuild

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
CURRENT, STREAM = 0, 0x5000      # the current device, and the handle of its current stream


class Tensor:
    """What the argument checks look at."""

    def __init__(self, shape, dtype=BF16, device="cuda:0", at=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.at = at if at is not None else 1 << 20

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.shape.numel()


class Library:
    """Records calls: name -> arguments of the last one."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls[name] = args
            return 0
        return call


@pytest.fixture
def ops(monkeypatch):
    mbuild.build()
    from mhc_hyper_connection_gb300 import _layer_ops
    monkeypatch.setattr(_layer_ops, "_lib", Library())
    monkeypatch.setattr(_layer_ops, "_current_device", lambda: CURRENT, raising=False)
    monkeypatch.setattr(_layer_ops, "_current_raw_stream", lambda index: STREAM + index)
    return _layer_ops


def _calls(ops, device):
    """Every launching call, with outputs and workspace given: (C function, call of `stream`)."""
    def t(*shape, d=BF16):
        return Tensor(shape, d, device)
    T, n, D, F = 3, 4, 64, 128
    ck = ops.Ckpt8(t(T, n, D, d=U8), t(T, n, 1, d=U8))
    x, res, post, comb = t(T, D), t(T, n, D), t(T, n, d=F32), t(T, n, n, d=F32)
    grads = {"grad_x": t(T, D), "grad_residual": t(T, n, D), "grad_post": t(T, n, d=F32), "grad_comb": t(T, n, n, d=F32)}
    w, wd, kept, ws = t(2, F, D), t(D, F), t(T, 2, F), t(1 << 20, d=U8)
    ffn = {"grad_x": t(T, D), "grad_w_gate_up": t(2, F, D), "grad_w_down": t(D, F)}
    return [("mhc_ckpt8_pack_run", lambda s: ops.ckpt8_pack(res, out=ck, stream=s)),
            ("mhc_ckpt8_restore_run", lambda s: ops.ckpt8_restore(ck, out=t(T, n, D), stream=s)),
            ("mhc_post_ckpt_run", lambda s: ops.hc_post_ckpt(x, res, post, comb, out=t(T, n, D), ckpt=ck, stream=s)),
            ("mhc_post_backward_run", lambda s: ops.hc_post_backward(t(T, n, D), x, res, post, comb, grads=grads, stream=s)),
            ("mhc_ffn_run", lambda s: ops.gated_ffn(x, w, wd, y=t(T, D), workspace=ws, stream=s)),
            ("mhc_ffn_backward_run", lambda s: ops.gated_ffn_backward(t(T, D), x, w, wd, kept, grads=ffn, workspace=ws,
                                                                      stream=s))]


@pytest.mark.parametrize("k", range(6))
def test_streams(ops, k):
    """A call runs on torch's current stream, a torch stream or a raw handle."""
    name, call = _calls(ops, "cuda:0")[k]
    for stream, want in ((None, STREAM), (77, 77), (type("S", (), {"cuda_stream": 99})(), 99)):
        call(stream)
        assert ops._lib.calls[name][-1] == want


@pytest.mark.parametrize("k", range(6))
@pytest.mark.parametrize("device", ["cpu", "cuda:1"])
def test_tensors_of_another_device(ops, k, device):
    """Neither host tensors nor those of a device that is not the current one
    reach the library, whatever stream is given."""
    _, call = _calls(ops, device)[k]
    for stream in (None, 77):
        with pytest.raises(ValueError):
            call(stream)
    assert not ops._lib.calls


@pytest.fixture
def binding(monkeypatch):
    """The binding of the mappings, its library replaced like that of `ops`."""
    mbuild.build()
    from mhc_hyper_connection_gb300 import _binding
    op = _binding.MhcPre(4, 64)                     # its handle comes from the real library
    record = Library()
    monkeypatch.setattr(_binding, "library", lambda: record)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: CURRENT)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: type("S", (), {"cuda_stream": STREAM + (getattr(device, "index", 0) or 0)})())
    _binding.record, _binding.op = record, op
    yield _binding
    monkeypatch.undo()
    op.close()


def _mapping_calls(b, device):
    def t(*shape, d=BF16):
        return Tensor(shape, d, device)
    T, n, D = 3, 4, 64
    x, phi, alpha, bias = t(T, n, D), t(24, n * D, d=F32), t(3, d=F32), t(24, d=F32)
    out = {"y": t(T, D), "h_post": t(T, n, d=F32), "inv_rms": t(T, d=F32), "h_mix": t(T, 24, d=F32)}
    return [("mhc_post_run", lambda s: b.hc_post(t(T, D), x, t(T, n, d=F32), t(T, n, n, d=F32), out=t(T, n, D), stream=s)),
            ("mhc_pre_run", lambda s: b.op.run(x, phi, alpha, bias, out, stream=s)),
            ("mhc_pre_sinkhorn_run", lambda s: b.op.run_composite(x, phi, alpha, bias, out, stream=s)),
            ("mhc_pre_backward_run", lambda s: b.op.backward(x, phi, alpha, None, t(T, D), t(T, n, d=F32), t(T, n, n, d=F32),
                                                             out, {}, stream=s))]


@pytest.mark.parametrize("k", range(4))
def test_mappings_on_their_device_and_others(binding, k, monkeypatch):
    """The pre-mapping and the post-mapping: the stream that the library gets,
    and no call for tensors of another device."""
    monkeypatch.setattr(Tensor, "element_size", lambda self: 1, raising=False)
    name, call = _mapping_calls(binding, "cuda:0")[k]
    for stream, want in ((None, STREAM), (77, 77), (type("S", (), {"cuda_stream": 99})(), 99)):
        call(stream)
        got = binding.record.calls[name][-1]
        assert getattr(got, "value", got) == want
    binding.record.calls.clear()
    for device in ("cpu", "cuda:1"):
        for stream in (None, 77):
            with pytest.raises(ValueError):
                _mapping_calls(binding, device)[k][1](stream)
    assert not binding.record.calls


def test_status_waits_for_the_current_stream(ops):
    """With and without a workspace the default is torch's current stream, not
    the legacy default stream, which does not order behind torch's others."""
    ws = Tensor((1024,), U8)
    for stream, want in ((None, STREAM), (77, 77), (0, None), (type("S", (), {"cuda_stream": 99})(), 99)):
        ops.gated_ffn_status(stream=stream)
        assert ops._lib.calls["mhc_ffn_status"] == (None, want)
    for stream, want in ((None, STREAM), (77, 77)):
        ops.gated_ffn_status(ws, stream=stream)
        assert ops._lib.calls["mhc_ffn_status"] == (ws.at, want)


def test_mapping_status_waits_for_the_current_stream(binding, monkeypatch):
    """As above for MhcPre.status, which reads the error word of a workspace:
    read on the legacy default stream it could be read before the run."""
    monkeypatch.setattr(Tensor, "element_size", lambda self: 1, raising=False)
    for stream, want in ((None, STREAM), (77, 77), (0, None)):
        binding.op.status({"workspace": Tensor((1024,), U8)}, stream=stream)
        assert binding.record.calls["mhc_pre_status"][-1].value == want


def test_run_without_tokens(binding):
    """x None stands for no tokens: the call still reaches the library."""
    binding.op.run(None, None, None, None, {"y": None}, stream=77)
    assert getattr(binding.record.calls["mhc_pre_run"][-1], "value", None) == 77
