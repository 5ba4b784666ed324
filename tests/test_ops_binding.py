"""What the operators' entry points refuse beside the contracts of each call: in
the binding, tensors whose elements are of another type than the call's, also where
the width is the same and the bytes would suffice; in the C ABI, outputs on top of
inputs that other rows are still to be read from."""

import pytest

import split_reduction_amd as sk
from tests.gpu_util import DEV, torch

A = 1 << 20  # an address; every call below is refused before any is used


class OnGpu:
    """A host tensor that says it is on the GPU: what the binding looks at."""

    is_cuda = True

    def __init__(self, a):
        self.a = a

    def __getattr__(self, name):
        return getattr(self.a, name)


def norm(Y=A, fmt="i8", **kw):
    a = {"X": A, "R": A, "G": A, "R_out": A, "y_scale": A, **kw}
    sk.skgemm_rmsnorm(a["X"], a["R"], a["G"], a["R_out"], Y, a["y_scale"], 4, 64, 1e-6, fmt)


def i8(fmt=None, **kw):
    a = {"Wq": A, "w_scale": A, "Xq": A, "x_scale": A, "C": A, **kw}
    sk.skgemm_i8(a["Wq"], a["w_scale"], a["Xq"], a["x_scale"], a["C"], 4, 64, 64, fmt)


def logprobs(fmt=None, **kw):
    names = ("logits", "tokens", "logprob", "entropy", "lse", "top_logprob", "top_ids")
    sk.skgemm_logprobs(*[({n: A for n in names} | kw)[n] for n in names], 4, 64, 16, logits_format=fmt)


def grad(fmt=None, **kw):
    names = ("logits", "tokens", "lse", "entropy", "g_logprob", "g_entropy", "d_logits")
    sk.skgemm_logprobs_grad(*[({n: A for n in names} | kw)[n] for n in names], 4, 64, logits_format=fmt)


# (call, argument, the wrong element type, arguments beside it)
WRONG = [
    *[(norm, n, ty, {}) for n in ("X", "R", "G", "R_out") for ty in ("float16", "int16", "float32")],
    *[(norm, "Y", ty, {"fmt": f}) for f, tys in (("bf16", ("float16", "int16", "uint8")), ("i8", ("float8_e4m3fn", "bfloat16")),
                                                 ("e4m3", ("int8", "float8_e5m2", "bfloat16"))) for ty in tys],
    *[(norm, "y_scale", ty, {}) for ty in ("float64", "int32", "bfloat16")],
    *[(i8, n, ty, {}) for n in ("Wq", "Xq") for ty in ("uint8", "float8_e4m3fn", "bfloat16")],
    *[(i8, n, ty, {}) for n in ("w_scale", "x_scale") for ty in ("float64", "int32")],
    *[(i8, "C", ty, {"fmt": f}) for ty in ("float16", "int32", "float64") for f in (None, "bf16", "f32")],
    (i8, "C", "float32", {"fmt": "bf16"}), (i8, "C", "bfloat16", {"fmt": "f32"}),
    *[(c, "logits", ty, {"fmt": f}) for c in (logprobs, grad) for ty in ("float16", "int32", "float64") for f in (None, "bf16", "f32")],
    *[(c, "tokens", ty, {}) for c in (logprobs, grad) for ty in ("int32", "float64")],
    *[(logprobs, n, ty, {}) for n in ("logprob", "entropy", "lse", "top_logprob") for ty in ("float64", "int32")],
    (logprobs, "top_ids", "float64", {}), (logprobs, "top_ids", "int32", {}),
    *[(grad, n, ty, {}) for n in ("lse", "entropy", "g_logprob", "g_entropy") for ty in ("float64", "int32")],
    (grad, "d_logits", "float16", {}), (grad, "d_logits", "float32", {}), (grad, "d_logits", "bfloat16", {"fmt": "f32"}),
]


@pytest.mark.parametrize("call,name,ty,more", WRONG)
def test_other_element_types_refused(call, name, ty, more):
    t = torch()
    a = t.zeros(4 * 64 * 8, dtype=t.uint8).view(getattr(t, ty)).view(4, -1)[:, :64].contiguous()  # bytes enough for each argument
    with pytest.raises(sk.SkgemmError) as e:
        call(**{name: OnGpu(a)}, **more)
    assert e.value.code == sk.SKGEMM_EINVAL and f"{name}: elements of torch.{ty}" in str(e.value), str(e.value)


@pytest.mark.gpu
def test_other_element_types_refused_on_the_gpu():
    """With whole buffers, of the same width as the call's."""
    t = torch()
    new = lambda *s, ty=t.float32: t.zeros(*s, dtype=ty, device=DEV)  # noqa: E731
    half, x, y, f = new(4, 64, ty=t.float16), new(4, 64, ty=t.bfloat16), new(4, 64, ty=t.int8), new(64)
    w, tok = new(64, 64, ty=t.int8), new(4, ty=t.int64)
    for call in (lambda: sk.skgemm_rmsnorm(half, None, None, None, y, f, 4, 64, 1e-6, "i8"),
                 lambda: sk.skgemm_rmsnorm(x, None, None, None, y, f, 4, 64, 1e-6, "e4m3"),
                 lambda: sk.skgemm_i8(w, f, y.view(t.float8_e4m3fn), f, x, 4, 64, 64),
                 lambda: sk.skgemm_i8(w, f, y, f, half, 4, 64, 64),
                 lambda: sk.skgemm_logprobs(half, tok, f, f, f, None, None, 4, 64),
                 lambda: sk.skgemm_logprobs_grad(half, tok, f, f, f, f, half, 4, 64)):
        with pytest.raises(sk.SkgemmError) as e:
            call()
        assert e.value.code == sk.SKGEMM_EINVAL and "elements of" in str(e.value)


def test_rmsnorm_sum_on_an_input_needs_its_stride():
    """Refused before any device work: the addresses are made up."""
    X, R, far = A, 1 << 24, 1 << 26

    def call(R_out, x_stride, r_stride, r_out_stride, r=R, T=3):
        return sk.lib().skgemm_rmsnorm(X, r, None, R_out, far, far, T, 64, 1e-6, 1, x_stride, r_stride, r_out_stride, 64, None)

    assert call(X, 0, 128, 128) == call(X, 256, 128, 128) == call(X, 128, 128, 256) == sk.SKGEMM_EINVAL
    assert call(R, 128, 0, 128) == call(R, 128, 256, 128) == call(R, 128, 128, 256) == sk.SKGEMM_EINVAL
    assert call(X, 256, 128, 128, r=None) == sk.SKGEMM_EINVAL


def test_scale_past_the_kernels_range_refused():
    """scale / log 2 has to be in FP32's range: beyond, every output was NaN."""
    f, b = sk.lib().skgemm_logprobs, sk.lib().skgemm_logprobs_grad
    for scale in (2.1e38, 3e38, 3.4e38):
        assert f(A, A, A, A, A, A, A, 2, 32, 4, scale, 0, 64, None) == sk.SKGEMM_EINVAL
        assert b(A, A, A, A, A, A, A << 1, 2, 32, scale, 0, 64, 64, None) == sk.SKGEMM_EINVAL
