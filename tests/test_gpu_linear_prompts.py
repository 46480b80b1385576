"""Prompts of linear_fwd on the GPU, beside tests/test_gpu_linear.py: what the outputs are rounded to, and every
walk and combine that the call's sizes choose, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from tests.linear_harness import HALF, TINY, Case, close, f64

pytestmark = pytest.mark.gpu

U = HALF[torch.bfloat16]
# P and the state enter the products that make an output as two bf16 terms: the first is cut off (it leaves less
# than 2^-7 of the value), the second rounds what is left (2^-8 of it).
TERMS = 2.0 ** -15


def _say(msg):
    print(msg, flush=True)


def _check_out(case, out, longest=None):
    """Outputs elementwise within one rounding, the terms' rest and the fp32 sums; and all together as far off as one
    rounding is: an error uniform in half a step to either side has a mean square of step^2 / 12."""
    o, S, oa, Sa = case.oracle()
    rows = int(case.cu[-1])
    got, o, oa = f64(out).reshape(o.shape)[:rows], o[:rows], oa[:rows]
    rel = close("out", got, o, oa, TERMS, longest or max(case.lengths), U, TINY[torch.bfloat16])
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(o), 1e-30))) - 7)
    want = np.sqrt((step ** 2).sum() / 12) / np.linalg.norm(o)
    # A sum of n squares of uniform errors is off by about sqrt(0.8 / n): 1 % at 10^4, and half as much of its root.
    assert o.size >= 10_000 and rel <= 1.05 * want, f"out: rel-L2 {rel:.3e}, one rounding makes {want:.3e}"
    return S, Sa


@pytest.mark.parametrize("H,kw", [
    (2, dict()), (2, dict(K=64)), (4, dict(V=64)), (4, dict(K=64, V=64)), (2, dict(state_dtype="bf16", k_first=True)),
    (2, dict(state="none")), (2, dict(state="dense", decay="head")), (4, dict(decay="none", H_qk=2)), (14, dict()),
    (28, dict(K=64, H_qk=4)),
], ids=str)
def test_outputs_are_rounded_once(H, kw):
    case = Case([300, 70], H=H, seed=H, **kw)
    _say(f"case H={H} {kw}")
    d = case.device()
    out, final = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    _check_out(case, out)
