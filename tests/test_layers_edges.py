"""The token operators at the edges of what they accept: extreme logits and
temperatures, buffers that a caller owns, sizes where a cost could run away.

Bounds as in test_layers: U = 2^-24 is the most an fp32 rounding is off,
`half` the same for an output's type."""
import pytest
import torch

from sign_muon_optimizer_momentum_b200 import layers
from test_layers import BF16, F32, U, distill_inputs, distill_reference, half, padded


def device_ms(f, reps=5):
    """The least time of a call on the device."""
    f()
    best = float("inf")
    for _ in range(reps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        begin.record()
        f()
        end.record()
        end.synchronize()
        best = min(best, begin.elapsed_time(end))
    return best


def distill_bounds(z, u, splits, t, top, ref):
    """What the losses by row and worker and the gradient may be off, from
    check_distill of test_layers."""
    _, R, D, logq, p, on = ref
    zd = z.double()
    spread = torch.where(on, (torch.where(on[:, None], zd, 0.0).amax(1)
                              - torch.where(on[:, None] & z.isfinite(), zd, float("inf")).amin(1)).clamp(min=0) / t, 0.0)
    uu = u.double() / t
    inf = float("inf")
    uspread = torch.where(on, torch.where(u.isfinite(), uu, -inf).amax(1) - torch.where(u.isfinite(), uu, inf).amin(1), 0.0)
    e_q = (4 * spread + 8 + z.shape[1] / 256 + 64) * U
    e_p = (4 * uspread + 8 + top) * U
    size = (p * logq.clamp(min=-1e30).abs()).sum(1) + torch.special.entr(p).sum(1).abs()
    e_row = t * t * (e_q + e_p + (e_p + 8 * U) * size + top * U * (size + spread) + 8 * U * (spread + 1)) + U * R.abs()
    e_loss, e_dz = [], torch.zeros_like(D)
    for a, b in zip(splits, splits[1:]):
        k = max(int(on[a:b].sum()), 1)
        e_loss.append((e_row[a:b].sum() + U * R[a:b].abs().sum()) / k)
        e = t / k * ((e_q[a:b, None] + 4 * U) * logq[a:b].exp() + (e_p[a:b, None] + 4 * U) * p[a:b])
        e_dz[a:b] = e + half(z.dtype) * (D[a:b].abs() + e) + 2.0 ** -126
    return torch.stack(e_loss), e_row, e_dz


def check_result(got, ref, bounds):
    """Losses by worker, by row, and the gradient, each within its bound."""
    for what, g, r, e in zip(("loss", "row_loss", "gradient"), got, ref, bounds):
        assert ((g.double() - r).abs() <= e).all(), what


MISALIGNED = [([700, 0, 1, 900, 300], 1100, 5, "holes"), ([1300, 40], 1030, 70, "plain"), ([3], 70001, 9, "twice")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shares,vocab,top,kind", MISALIGNED)
def test_distill_rows_at_any_address(cuda_lib, dtype, shares, vocab, top, kind):
    """Logits off 16 bytes, whose rows a block takes from several workers."""
    z, ids, u, splits = distill_inputs(shares, vocab, top, dtype, kind)
    z = padded(z, 3, offset=1)
    ref = distill_reference(z, ids, u, splits, 2.0)
    bounds = distill_bounds(z, u, splits, 2.0, top, ref)
    check_result(layers.distill_loss_and_grad(z, ids, u, len(shares), splits, temperature=2.0), ref, bounds)
    over = layers.distill_loss_and_grad(z, ids, u, len(shares), splits, temperature=2.0, out=z)
    assert over[2] is z
    check_result(over, ref, bounds)


@pytest.mark.gpu
def test_distill_misaligned_gradient_grows_with_its_rows(cuda_lib):
    """Ten times the rows of one worker take about ten times as long: what a
    row costs does not depend on how many rows its worker has."""
    def ms(n):
        z = padded(torch.zeros(n, 1100, dtype=BF16, device="cuda"), 1, offset=1)
        ids, u = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
        out = torch.empty(n, 1101, dtype=BF16, device="cuda")[:, 1:]
        return device_ms(lambda: layers.distill_loss_and_grad(z, ids, u, out=out))
    assert ms(200000) <= 14 * ms(20000)
