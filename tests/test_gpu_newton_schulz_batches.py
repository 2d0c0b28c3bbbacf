"""Newton-Schulz batches that are longer than the scratch holds at a time, and polynomials at the number format's ends."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

pytestmark = pytest.mark.gpu


def part(M, N):
    """Matrices of a batch that are worked off together: from this many on the scratch stays the same."""
    most = mp.mpgemm_run_newton_schulz_workspace(60000, M, N)
    lo, hi = 1, 60000
    while lo < hi:
        mid = (lo + hi) // 2
        if mp.mpgemm_run_newton_schulz_workspace(mid, M, N) == most:
            hi = mid
        else:
            lo = mid + 1
    return lo


# a side up to 128, single steps, groups, groups with the sum over the long side split; an odd and an even number of
# exchanges of the buffers in a part; a last part that is shorter
@pytest.mark.parametrize("M,N,steps", [(33, 40, 5), (33, 40, 4), (600, 700, 5), (1300, 600, 5), (600, 1300, 2), (192, 1280, 5)])
def test_more_than_one_part(M, N, steps):
    n = part(M, N)
    B = n + n // 20 + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + steps)
    x = torch.empty(B, M, N, dtype=torch.bfloat16, device="cuda")
    for i in range(0, B, 1000):
        x[i:i + 1000] = torch.randn(min(1000, B - i), M, N, generator=g, device="cuda")
    y = mp.newton_schulz(x, steps=steps)
    assert torch.isfinite(y).all()
    cut = n // 2 + 1   # both pieces in one go each
    assert torch.equal(y[:cut], mp.newton_schulz(x[:cut], steps=steps))
    assert torch.equal(y[cut:], mp.newton_schulz(x[cut:], steps=steps))
    for b in (0, n - 1, n, B - 1):
        assert torch.equal(y[b], mp.newton_schulz(x[b], steps=steps))
    mp.newton_schulz(x, steps=steps, out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("M,N", [(40, 60), (150, 170)])
def test_huge_coefficients(M, N):
    """Multiples of X, up to where the squares of its singular values leave fp32: the call refuses those."""
    g = torch.Generator()
    g.manual_seed(M)
    x = torch.randn(M, N, generator=g).to(torch.bfloat16)
    unit = x.double() / torch.linalg.vector_norm(x.double())
    for steps, a in ((1, 1e30), (2, 1e15), (3, 1e8), (4, 1e6)):
        y = mp.newton_schulz(x.cuda(), steps=steps, coeffs=(a, 0.0, 0.0)).double().cpu()
        want = float(torch.tensor(a)) ** steps * unit
        off = torch.linalg.vector_norm(y - want) / torch.linalg.vector_norm(want)
        assert off <= 2.0 ** -8 * 1.125, (steps, a)
    for steps, a in ((2, 1e20), (3, 1e12), (6, 1e6)):
        with pytest.raises(mp.MpgemmError) as e:
            mp.newton_schulz(x.cuda(), steps=steps, coeffs=(a, 0.0, 0.0))
        assert e.value.status == mp.MPGEMM_ERR_UNSUPPORTED
