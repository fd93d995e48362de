"""The binding of the stored operands without a GPU: tensors that only look like
CUDA ones, and the library's entry points recorded instead of called."""
import pytest
import torch


class Fake:
    """What the binding reads of a CUDA tensor, over a CPU one (never computed
    with)."""

    def __init__(self, t, device=0):
        self.t, self.device_index = t, device

    is_cuda = True
    shape = property(lambda self: self.t.shape)
    dtype = property(lambda self: self.t.dtype)
    itemsize = property(lambda self: self.t.element_size())

    def stride(self, *i):
        return self.t.stride(*i)

    nbytes = property(lambda self: self.t.nbytes)

    def numel(self):
        return self.t.numel()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def data_ptr(self):
        return self.t.data_ptr()

    def get_device(self):
        return self.device_index


@pytest.fixture
def b(lib_path, monkeypatch):
    from dense_gemm_tiled_gb300 import binding
    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    monkeypatch.setattr(binding, "_lib", Recorder())
    monkeypatch.setattr(binding, "_current_stream", lambda dev: 0)
    binding.calls = calls
    yield binding
    del binding.calls


def mx(b, rows, cols, fmt, device=0):
    need = {"fp4": -(-cols // 32) * 16, "int8": -(-cols // 16) * 16, "fp4_e4m3": -(-cols // 32) * 16}
    blocks = -(-cols // (16 if fmt == "fp4_e4m3" else 32))
    scales = -(-rows // 128) * -(-blocks // 4) * 512
    return b.Mx(Fake(torch.zeros((rows, need[fmt]), dtype=torch.uint8), device),
                Fake(torch.zeros(scales, dtype=torch.uint8), device), fmt, rows, cols)


def every_call(b, Q8, B, A, device=0):
    """Each entry point once, with the stored operands Q8 (int8) and A, B (fp4)."""
    t = lambda *s: Fake(torch.zeros(s, dtype=torch.float16), device)  # noqa: E731
    X, Y = t(Q8.rows, Q8.cols), t(Q8.rows, Q8.cols)
    return {
        "quantize": lambda: b.mx_quantize(X, Q8),
        "dequantize": lambda: b.mx_dequantize(Q8, Y),
        "act": lambda: b.mx_act_backward(X, Q8, Y),
        "mixed": lambda: b.gemm_mx(t(5, B.cols), B, t(5, B.rows), transB=True),
        "mx4": lambda: b.gemm_mx(A, B, t(A.rows, B.rows)),
    }


NAMES = ["quantize", "dequantize", "act", "mixed", "mx4"]


@pytest.mark.parametrize("name", NAMES)
def test_replaced_storage_is_used(b, name):
    """`.data` of a stored tensor replaced after the Mx was made (as moving or
    offloading a module does): the next call gets the new address."""
    Q8, B, A = mx(b, 130, 70, "int8"), mx(b, 40, 96, "fp4"), mx(b, 7, 96, "fp4")
    call = every_call(b, Q8, B, A)[name]
    call()
    old = b.calls[-1][1]
    new = []
    for Q in (Q8, B, A):
        for f in (Q.codes, Q.scales):
            f.t = f.t.clone()
            new.append(f.t.data_ptr())
    call()
    got = b.calls[-1][1]
    assert got != old
    for k, addresses in {"quantize": new[:2], "dequantize": new[:2], "act": new[:2],
                         "mixed": new[2:4], "mx4": new[2:6]}.items():
        if k == name:
            assert all(p in got for p in addresses)
    # a tensor in the other's place
    for Q in (Q8, B, A):
        Q.codes = Fake(Q.codes.t.clone())
    call()
    used = [Q.codes.data_ptr() for Q in {"mixed": (B,), "mx4": (A, B)}.get(name, (Q8,))]
    assert all(p in b.calls[-1][1] for p in used)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("what", ["rows", "bytes", "stride", "scales", "host", "type"])
def test_replaced_storage_that_does_not_fit_is_refused(b, name, what):
    Q8, B, A = mx(b, 130, 70, "int8"), mx(b, 40, 96, "fp4"), mx(b, 7, 96, "fp4")
    call = every_call(b, Q8, B, A)[name]
    for Q in (Q8, B, A):
        if what == "rows":
            Q.codes.t = Q.codes.t[:-1]
        elif what == "bytes":
            Q.codes.t = Q.codes.t[:, :-16].contiguous()
        elif what == "stride":
            Q.codes.t = Q.codes.t.t().contiguous().t()
        elif what == "scales":
            Q.scales.t = Q.scales.t[:-1]
        elif what == "host":
            Q.scales = Fake(Q.scales.t.clone(), -1)
            Q.scales.is_cuda = False  # (a host tensor in its place)
        else:
            Q.codes.t = Q.codes.t.short()
    done = len(b.calls)
    with pytest.raises(TypeError if what == "type" else ValueError):
        call()
    assert len(b.calls) == done


@pytest.mark.parametrize("name", NAMES)
def test_operands_of_two_devices_are_refused(b, name):
    for dev in (0, 1):
        call = every_call(b, mx(b, 130, 70, "int8", dev), mx(b, 40, 96, "fp4", dev),
                          mx(b, 7, 96, "fp4", dev), dev)[name]
        call()
        done = len(b.calls)
        call = every_call(b, mx(b, 130, 70, "int8", dev), mx(b, 40, 96, "fp4", dev),
                          mx(b, 7, 96, "fp4", dev), 1 - dev)[name]
        with pytest.raises(ValueError):
            call()
        assert len(b.calls) == done


def test_every_tensor_is_on_the_device(b):
    t = lambda *s, dev=0, dt=torch.float16: Fake(torch.zeros(s, dtype=dt), dev)  # noqa: E731
    Q, B = mx(b, 130, 70, "int8"), mx(b, 40, 96, "fp4")
    bad = [
        lambda: b.mx_quantize(t(130, 70), Q, act="relu", Y=t(130, 70, dev=1)),
        lambda: b.mx_act_backward(t(130, 70), Q, t(130, 70, dev=1)),
        lambda: b.mx_act_backward(t(130, 70), Q, t(130, 70),
                                  dbias=t(70, dev=1, dt=torch.float32)),
        lambda: b.gemm_mx(t(5, 96, dev=1), B, t(5, 40), transB=True),
        lambda: b.gemm_mx(t(5, 96), B, t(5, 40), transB=True, bias=t(40, dev=1)),
        lambda: b.gemm_mx(mx(b, 5, 96, "fp4", 1), B, t(5, 40)),
        lambda: b.Mx(Q.codes, Fake(Q.scales.t, 1), "int8", 130, 70),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not b.calls


def test_scalars_that_gemm_takes(b):
    """alpha, beta and mult as Python numbers, numpy scalars and 0-d tensors;
    sizes as numpy integers."""
    import numpy as np
    t = lambda *s: Fake(torch.zeros(s, dtype=torch.float16))  # noqa: E731
    Q, B, A = mx(b, np.int64(130), np.int32(70), "int8"), mx(b, 40, 96, "fp4"), mx(b, 7, 96, "fp4")
    assert type(Q.rows) is int and type(Q.cols) is int
    for half in (0.5, np.float32(0.5), np.float64(0.5), torch.tensor(0.5)):
        b.mx_quantize(t(130, 70), Q, mult=half)
        b.gemm_mx(t(5, 96), B, t(5, 40), transB=True, alpha=half, beta=half)
        b.gemm_mx(A, B, t(7, 40), alpha=half, beta=half)
        for (name, args), n in zip(b.calls[-3:], (1, 2, 2)):
            given = [v for v in args if type(v) is float]
            assert given == [0.5] * n, name
    assert all(type(v) in (int, float, type(None)) for _, args in b.calls for v in args)


def test_plain_tensors_in_a_stored_operands_place(b):
    t = lambda *s: Fake(torch.zeros(s, dtype=torch.float16))  # noqa: E731
    B = mx(b, 40, 96, "fp4")
    for call in (lambda: b.gemm_mx(t(5, 96), t(96, 40), t(5, 40)),
                 lambda: b.gemm_mx(B, t(96, 40), t(40, 40)),
                 lambda: b.mx_quantize(t(4, 8), t(4, 8)), lambda: b.mx_dequantize(t(4, 8), t(4, 8)),
                 lambda: b.mx_act_backward(t(4, 8), t(4, 8), t(4, 8))):
        with pytest.raises(TypeError, match="stored operand"):
            call()
    assert not b.calls
