"""Numbers that the int8 cache's kernels and formulas rest on, checked without a GPU."""
import os
import re

import numpy as np

from oracle import int8 as I

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_kv_cache_tq_gb300", "csrc")


def test_polynomials_of_sine_and_cosine():
    """The coefficients in the source, as fp32 holds them, evaluated in 64 bits over an eighth of a turn, against the
    errors that the source states."""
    text = open(os.path.join(CSRC, "tq_int8_rows.cu")).read()
    stated = re.search(r"sine ([\d.e-]+) relative, cosine\n?/*\s*([\d.e-]+)\)", text)
    sine, cosine = (re.search(rf"const float {p} = (.*);", text).group(1) for p in ("ps", "pc"))
    numbers = lambda line: [float(np.float32(x)) for x in re.findall(r"(-?[\d.]+(?:e-?\d+)?)f\b", line)]  # noqa: E731
    t = np.linspace(0, np.pi / 4, 1 << 20)[1:]
    u = t * t
    s, c = np.polyval(numbers(sine), u), np.polyval(numbers(cosine), u)
    assert len(numbers(sine)) == 3 and len(numbers(cosine)) == 4
    assert np.abs((t + t * u * s) / np.sin(t) - 1).max() <= float(stated.group(1)) <= 1e-8
    assert np.abs(1 + u * c - np.cos(t)).max() <= float(stated.group(2)) <= 1e-8


def test_codes_and_scales_by_hand():
    # 0.635 / binary16(0.01) = 63.49; -127 by 1.27 / binary16(0.01) = 126.97; ties go to the even code
    c, s = I.quantise(np.array([[-1.27, 0.635, 0.0, 0.01, 1.27, -0.004], [31.75, 0.125, 0.375, 0.625, -0.125, -0.375]]))
    assert s.dtype == np.float16 and c.dtype == np.int8
    assert list(s) == [np.float16(0.01), np.float16(0.25)]
    assert list(c[0]) == [-127, 63, 0, 1, 127, 0]
    assert list(c[1]) == [127, 0, 2, 2, 0, -2]
