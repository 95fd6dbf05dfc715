"""The polynomial of softplus (csrc/selective.hpp): its constants as written there, in 64 bits, against log(1 + e^-x) over
its whole range, within the error that its comment states."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sketched_recurrent_state_amd", "csrc",
                      "selective.hpp")


def test_polynomial():
    with open(SOURCE) as f:
        text = f.read()
    stated = float(re.search(r"largest relative error is the least \(([0-9.e-]+),", text).group(1))
    body = text[text.index("float softplus(float x)"):]
    body = body[:body.index("\n}\n")]
    top, nxt = re.search(r"p = fmaf\(q, ([0-9.]+)f, ([0-9.]+)f\);", body).groups()
    consts = [top, nxt] + re.findall(r"p = fmaf\(q, p, ([0-9.]+)f?\);", body)
    assert len(consts) == 5 and float(consts[-1].rstrip("f")) == 1
    e = np.concatenate([np.logspace(-12, -3, 10000), np.linspace(1e-3, 1, 1000000)])
    s = e / (2 + e)
    p = np.zeros_like(s)
    for c in consts:
        p = p * s * s + float(np.float32(c))
    off = np.abs(2 * s * p / np.log1p(e) - 1).max()
    assert off <= stated <= 1.05 * off, (off, stated)
