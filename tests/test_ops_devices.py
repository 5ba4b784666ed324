"""Tensors of another GPU than the current one, where the call would be launched, are
refused: every argument of the calls that take many, whether or not a stream is given."""

import pytest

import split_reduction_amd as sk
from tests.gpu_util import torch
from tests.test_ops_binding import OnGpu

A = 1 << 20  # an address; no call below reaches the library


class OnAnother(OnGpu):
    def get_device(self):
        return 1


def tensor(size, ty="bfloat16"):
    t = torch()
    return OnAnother(t.zeros(size, dtype=getattr(t, ty)))


ROPE = {"X": ((4, 128),), "G": ((64,),), "inv_freq": ((32,), "float32"), "positions": ((4,), "int64"), "Y": ((4, 128),)}
APPEND = {"Q": ((4, 128),), "K": ((4, 64),), "V": ((4, 64),), "Gq": ((64,),), "Gk": ((64,),), "inv_freq": ((32,), "float32"),
          "positions": ((4,), "int64"), "slots": ((4,), "int64"), "Q_out": ((4, 128),), "K_cache": ((3, 16, 1, 64),), "V_cache": ((3, 16, 1, 64),)}
ATTENTION = {"Q": ((4, 128),), "K_cache": ((3, 16, 1, 64),), "V_cache": ((3, 16, 1, 64),), "page_table": ((2, 2), "int32"),
             "kv_len": ((2,), "int32"), "q_start": ((3,), "int32"), "O": ((4, 128),), "lse": ((4, 2), "float32")}
CALLS = [(sk.skgemm_rope, ROPE, (4, 2, 64, 64)), (sk.skgemm_rope_append, APPEND, (4, 2, 1, 64, 3, 16, 64)),
         (sk.skgemm_paged_attention, ATTENTION, (4, 2, 2, 2, 1, 64, 3, 16, 2, 0.125))]


@pytest.mark.parametrize("stream", [0, None])
@pytest.mark.parametrize("call,args,sizes,name", [(c, a, s, n) for c, a, s in CALLS for n in a])
def test_tensor_on_another_gpu_refused(monkeypatch, call, args, sizes, name, stream):
    t = torch()
    for what in ("_raw_stream", "_device", "_gpus"):
        monkeypatch.setattr(sk, what, None)
    monkeypatch.setattr(t.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(t.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(t._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(sk, "lib", lambda: pytest.fail("the library was reached"))
    with pytest.raises(sk.SkgemmError) as e:
        call(*[tensor(*args[n]) if n == name else A for n in args], *sizes, stream=stream)
    assert e.value.code == sk.SKGEMM_EINVAL and str(e.value).count(f"{name}: a tensor on GPU 1"), str(e.value)
