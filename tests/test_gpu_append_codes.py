"""The E4M3 codes that skgemm_rope_append stores: of value / scale in FP32, to nearest
even, for every bf16 value."""

import numpy as np
import pytest

import split_reduction_amd as sk
from oracle import formats as F
from tests.gpu_util import DEV, log, torch

# Products with the rounded reciprocal of all but the last two fall on the other side
# of a border between two codes for some values.
SCALES = [0.48, 0.03197338059544563, 0.0546875, 0.03, 0.3, 0.12364130467176437, 0.0019318953854963183, 0.11, 0.125]


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("scale", SCALES)
def test_codes_are_of_the_quotient(scale, order):
    t = torch()
    log(f"codes of every bf16 value / {scale}")
    T, H, D, page = 256, 2, 128, 16
    x = t.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(t.bfloat16)
    with np.errstate(all="ignore"):
        quotient = x.float().numpy() / np.float32(scale)
    nan = np.isnan(quotient)
    want = F.e4m3_value(F.f32_to_e4m3_rne(np.clip(np.where(nan, 0, quotient), -448, 448)))
    rows = x.view(T, H * D).to(DEV)
    other = 0.25
    shape = (T // page, page, H, D) if order == "token" else (T // page, H, page, D)
    for scales in ((scale, other), (other, scale)):
        kc, vc = (t.zeros(shape, dtype=t.uint8, device=DEV) for _ in "kv")
        if order == "head":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        sk.skgemm_rope_append(None, rows, rows, None, None, None, None, t.arange(T, device=DEV), None, kc, vc, T, 0, H, D, T // page, page,
                              0, k_scale=scales[0], v_scale=scales[1])
        t.cuda.synchronize()
        codes = (kc if scales[0] == scale else vc).contiguous().cpu().numpy().reshape(-1)
        with np.errstate(invalid="ignore"):
            got = F.e4m3_value(codes)
        assert np.isnan(got[nan]).all()
        wrong = np.nonzero((got != want) & ~nan)[0]
        assert len(wrong) == 0, (len(wrong), quotient[wrong[:4]], got[wrong[:4]], want[wrong[:4]])
