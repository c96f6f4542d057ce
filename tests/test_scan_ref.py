"""The comparison that the scan's GPU tests use (no GPU): what it lets through and what it does not, at their lengths."""
import numpy as np
import pytest
import torch

import scan_ref as ref

LENS = {"cut": [700, 0, 5, 400, 130], "uneven": [3, 1, 0, 40] * 2 + [4100] + [2] * 8, "long": [9000]}


@pytest.fixture(scope="module", params=LENS)
def case(request):
    lens = LENS[request.param]
    s = ref.inputs(lens, 6, 2, 16, torch.float32, device="cpu")
    return lens, ref.scan(s, lens), ref.scan(s, lens, np.float32)


def test_fp32_passes(case):
    """The formulas in fp32, token by token, stay within a half of the bounds."""
    lens, want, single = case
    for name, w in want.items():
        assert ref.off(name, single[name], w, lens) <= 0.5 * ref.BOUND.get(name, ref.BACKWARD), name
        for dtype in (torch.float32, torch.bfloat16):
            ref.check(name, torch.from_numpy(w).to(dtype), w, lens)


def test_wrong_outputs_do_not(case):
    """Zeroed, off by a hundredth, or either of them in one part alone; in 32 bits and in bf16."""
    lens, want, _ = case
    for name, w in want.items():
        where = list(ref.parts(name, w.shape, lens))
        where = [p for p in where if np.any(w[p])]
        assert where, name
        for p in (slice(None), where[0], where[len(where) // 2], where[-1]):
            for factor in (0.0, 0.99, 1.01, float("nan")):
                bad = w.copy()
                bad[p] *= factor
                for dtype in (torch.float32, torch.bfloat16):
                    with pytest.raises(AssertionError):
                        ref.check(name, torch.from_numpy(bad).to(dtype), w, lens)
