"""What the packed SSD kernels keep of 32 bits: outputs in bf16 are the 64-bit values rounded once, and nothing else.

Every product on the matrix cores has one factor that is bf16 already and one in parts.  Two parts leave out 2^-16 of a
value at most, three 2^-24.  The decays' logarithms are summed without loss that counts, their exponentials are good to
2^-22 and the step sizes' to 2^-21; a sum of up to 512 terms in fp32 rounds by 2^-24 each, 2^-15 of the magnitudes at worst.
"""
import pytest

import packed_ref as R
from test_packed_gpu import BF, SSD, f64, ssd_case, ssd_ref, ssm, T, within

pytestmark = pytest.mark.gpu

# what stands before the last rounding, of the sum of the magnitudes: 2^-16 (parts) + 2^-15 (sums) + 2^-19 (step, decay)
REST = 2.0 ** -14


@pytest.mark.parametrize("k", range(len(SSD)))
def test_y_is_rounded_once(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    ref, _, mag = ssd_ref(c, cul, first, how)
    y = ssm().ssd_packed_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], c["cu"], c["bias"], c["D"], state=state,
                             state_idx=idx, has_state=has, **kw)
    torch.cuda.synchronize()
    inside = slice(cul[0], cul[-1])
    within(y[inside], (BF * ref.abs() + REST * mag + 1e-30)[inside], ref[inside], "y")


@pytest.mark.parametrize("k", range(len(SSD)))
def test_gradients_are_rounded_once(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    H, N = c["x"].shape[1], c["B"].shape[2]
    dy = r(rows, H, 64, dtype=torch.bfloat16)
    dl = r(len(cul) - 1, H, 64, N, scale=0.3)
    wide = [f64(c[n]) for n in ("x", "dt", "A", "B", "C", "bias", "D")]
    ref = R.ssd_grads(*wide, cul, first, f64(dy), f64(dl), **how)
    # with every factor's magnitude the same formulas sum the magnitudes of the terms
    big = [t if t is None or n in "dt A bias" else t.abs() for n, t in zip(("x", "dt", "A", "B", "C", "bias", "D"), wide)]
    mag = R.ssd_grads(*big, cul, first.abs(), f64(dy).abs(), f64(dl).abs(), **how)
    got = ssm().ssd_packed_bwd(c["x"], c["dt"], c["A"], c["B"], c["C"], dy, c["cu"], c["bias"], c["D"], state=state,
                               state_idx=idx, has_state=has, dstate_out=dl, **kw)
    torch.cuda.synchronize()
    inside = slice(cul[0], cul[-1])
    for n in ("dx", "dB", "dC"):
        within(got[n][inside], (BF * ref[n].abs() + REST * mag[n] + 1e-30)[inside], ref[n][inside], n)
