"""A comparison that a NaN or infinity in the wrong place fails."""
import torch


def check(got, want, tol, what):
    got, want = got.to(torch.float64).cpu(), want.to(torch.float64).cpu()
    assert got.shape == want.shape, what
    good = ((got - want).abs() <= tol) | (got == want) | (got.isnan() & want.isnan())
    assert bool(good.all()), f"{what}: {int((~good).sum())} of {good.numel()} off, {int(got.isnan().sum())} NaN, worst " \
        f"{float((got - want).abs().nan_to_num(0, 0).max())} at tolerance {float(torch.as_tensor(tol).max())}"
