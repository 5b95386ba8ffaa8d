"""The exponential that the key weights take on the FMA pipe, restated step by
step in fp32 with the constants of the source: its error is what is stated
there.  Host-only."""

import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_psa_b200",
                   "csrc", "sm100.cuh")
f32 = np.float32


def _constants():
    body = open(SRC).read().split("void exp2_parts(")[1].split("\n}\n")[0]
    bias = f32(re.search(r"kBias = ([\d.]+)f", body).group(1))
    lines = re.findall(r"ffma2\(p0, p1, (.*?)\);", body)
    first = re.findall(r"([\d.]+)f\b", lines[0])
    return bias, [f32(first[0]), f32(first[2])] + [f32(re.findall(r"([\d.]+)f\b", x)[0]) for x in lines[1:]]


def _exp2(x):
    fma = lambda a, b, c: (a.astype(np.float64) * b + np.float64(c)).astype(f32)  # noqa: E731
    bias, c = _constants()
    x = np.clip(x, f32(-126), f32(128))
    t = (x + bias).astype(f32)
    f = ((bias - t).astype(f32) + x).astype(f32)
    p = fma(np.full_like(f, c[0]), f, c[1])
    for k in c[2:]:
        p = fma(p, f, k)
    return p.astype(np.float64) * (t.view(np.uint32) << np.uint32(23)).view(f32)


def test_error_is_the_stated_one():
    assert len(_constants()[1]) == 6
    for lo in (-0.5, 0.25, -20.0, -100.0, 126.0):
        x = (np.arange(0, 1 << 24, 7) * 2.0 ** -24 + lo).astype(f32)
        e = _exp2(x) / np.exp2(x.astype(np.float64)) - 1
        assert -1.05e-7 < e.min() and e.max() < 2.15e-7 and abs(e.mean() - 5e-8) < 1e-8
    x = np.arange(-126, 128).astype(f32)
    assert np.abs(_exp2(x) / np.exp2(x.astype(np.float64)) - 1).max() < 1.2e-7


def test_ends_of_the_range():
    x = np.array([-1e30, -200, -126, 127.5, 127.51, 128, 1e30], f32)
    got = _exp2(x)
    assert (np.abs(got[:3] / 2.0 ** -126 - 1) < 1.2e-7).all()
    assert np.isfinite(got[3]) and np.isinf(got[4:]).all()
