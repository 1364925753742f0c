"""The polynomial of the scan's softplus, with the coefficients that dl_ssm.h holds (no
GPU needed): artanh(s) / s in w = s^2 <= 1/9, off by no more than the 2^-27.7 that is
stated there."""
import os
import re

import numpy as np

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_state_update_amd", "csrc",
                      "dl_ssm.h")


def coefficients():
    body = re.search(r"float softplus\(.*?\n}", open(HEADER).read(), re.S).group()
    first, = re.findall(r"float p = ([\d.]+)f;", body)
    rest = re.findall(r"p = fmaf\(p, w, ([\d.]+)f\);", body)
    return [np.float32(c).astype(np.float64) for c in (first, *rest)]  # of w^4 ... 1


def test_polynomial():
    c = coefficients()
    assert len(c) == 5 and c[-1] == 1
    w = np.linspace(0, 1 / 9, 1 << 18)
    series = sum(w ** k / (2 * k + 1) for k in range(30))  # (1/9)^30 / 61 is left
    off = np.abs(np.polyval(c, w) / series - 1)
    assert off.max() <= 2.0 ** -27.7, np.log2(off.max())


def test_no_other_with_a_constant_of_one_is_much_better():
    """Five points where the error of the committed one changes sign, and is 2^-27.8 or
    more at each: any other of this form is off by as much at one of them."""
    w = np.linspace(0, 1 / 9, 1 << 18)
    series = sum(w ** k / (2 * k + 1) for k in range(30))
    off = np.polyval(coefficients(), w) / series - 1
    runs = np.split(off, np.flatnonzero(np.diff(np.sign(off))) + 1)
    assert sum(np.abs(r).max() >= 2.0 ** -27.8 for r in runs) >= 5
