"""c128_build_cos_sin against angles of 60 digits: how far an angle may be off, near and far."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from deepseek_v4_sparse_c128_gb300 import binding

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def steps(width, theta=10000.0, scaling="none", factor=1.0, original_positions=65536, beta_fast=32.0, beta_slow=1.0, magnitude=1.0):
    """(radians per position of each pair, the same without the scaling)."""
    getcontext().prec = 60
    ln = Decimal(theta).ln()

    def pair(turns):
        return width * (Decimal(original_positions) / (2 * PI * Decimal(turns))).ln() / (2 * ln)
    low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), width - 1)
    out, plain = [], []
    for i in range(width // 2):
        f = (-ln * 2 * i / width).exp()
        plain.append(f)
        if scaling == "linear":
            f = f / Decimal(factor)
        if scaling == "yarn":
            g = min(max(Decimal(i - low) / max(Decimal(high - low), Decimal("0.001")), Decimal(0)), Decimal(1))
            f = f * (1 - g) + f / Decimal(factor) * g
        out.append(f)
    return out, plain


@pytest.mark.parametrize("width", [64, 96, 512])
@pytest.mark.parametrize("rope", [
    dict(), dict(theta=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="linear", factor=0.3),
    dict(scaling="yarn", factor=16.0, magnitude=1.2772588722239782), dict(theta=1e6, scaling="yarn", factor=40.0, original_positions=4096)],
    ids=lambda r: "-".join(str(v) for v in r.values()) or "plain")
def test_angles(width, rope):
    f, plain = steps(width, **rope)
    mag = rope.get("magnitude", 1.0)
    for first in (0, 1000, (1 << 18) - 1, (1 << 24) + 3, (1 << 32) - 3):
        table = torch.empty(3, width, device="cuda")
        binding.build_cos_sin(binding.rope(**rope), first, table)
        got = table.double().cpu().numpy()
        for row in range(3):
            turns = [(first + row) * x / (2 * PI) for x in f]
            angle = np.array([float((t - int(t)) * 2 * PI) for t in turns])
            most = np.array([max(float(t), float((first + row) * x / (2 * PI))) for t, x in zip(turns, plain)])
            off = abs(mag) * (2.0 ** -30 + 2.0 ** -46 * most)
            for part, want in ((got[row, :width // 2], mag * np.cos(angle)), (got[row, width // 2:], mag * np.sin(angle))):
                assert (np.abs(part - want) <= off + 2.0 ** -22 * np.abs(want)).all(), (first, row, np.max(np.abs(part - want) / off))
