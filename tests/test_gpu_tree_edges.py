"""pa_decode_tree where its tiles and weights meet their limits: values that are not finite over several checked tiles,
weights next to a rounding border, a scale of zero, unserved sequences."""
import math
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from oracle import tree as otree  # noqa: E402
from tree_harness import Batch, check  # noqa: E402

pytestmark = pytest.mark.gpu


def repeated(b, times, device):
    """The batch's only sequence `times` times over, all reading the same blocks: several whole items for every CTA."""
    x = b.gpu(device)
    for n in ("block_tables", "q", "mask"):
        if getattr(x, n) is not None:
            setattr(x, n, getattr(x, n).repeat(times, *[1] * (getattr(x, n).dim() - 1)))
    x.context_lens, x.N = x.context_lens.repeat(times), b.new[0] * times
    x.query_starts = torch.arange(times + 1, dtype=torch.int32, device=device) * b.new[0]
    return x


@pytest.mark.parametrize("heads", [(4, 2, 256, "bf16"), (8, 1, 256, "f16"), (1, 1, 256, "bf16"), (8, 1, 128, "bf16"),
                                   (1, 1, 128, "f16"), (8, 8, 64, "bf16"), (1, 1, 64, "f32")])
@pytest.mark.parametrize("prefix,new", [(63, 256), (40, 150), (0, 130)])
def test_values_in_three_to_five_checked_tiles(pa, cuda_device, heads, prefix, new):
    """One element of V infinite in every checked tile, each in a column of its own: those columns of the rows that
    attend it, and nothing else; alone and with rings that wrap around within a CTA's items."""
    H, G, d, t = heads
    b = Batch(50 + new, [prefix], [new], H, G, d, t, kind="any")
    nodes = sorted({min(new - 1, max(0, tile * 64 + off - prefix)) for tile, off in zip(range(5), (63, 3, 17, 40, 62))})
    for c, node in enumerate(nodes):
        row = torch.randn(G, d).to(b.dtype)
        row[:, 7 * c + 3] = float("-inf") if c % 2 else float("inf")
        b.set_row(0, prefix + node, v=row)
    with np.errstate(invalid="ignore"):
        ref = b.reference()
    allow = np.where(np.isfinite(b.allow), b.allow, 0.0)
    seen = np.array([otree.unpack_row(r, new) for r in b.mask.tolist()])
    for c, node in enumerate(nodes):
        assert (np.isinf(ref[:, :, 7 * c + 3]) == seen[:, node, None]).all()
    finite = np.isfinite(ref)
    for times in (1, 60):
        x = repeated(b, times, cuda_device)
        for out_dtype in (b.dtype, torch.float32):
            out = x.run(pa, out_dtype=out_dtype).cpu()
            ok, want = np.tile(finite, (times, 1, 1)), np.tile(ref, (times, 1, 1))
            assert (out.double().numpy()[~ok] == want[~ok]).all(), f"{heads} {new} x {times}"
            check(torch.where(torch.from_numpy(ok), out, torch.zeros_like(out)), np.where(ok, want, 0.0),
                  f"{heads} {new} x {times}", allow=np.tile(allow, (times, 1, 1)))
    assert pa.pa_get_error() == 0


@pytest.mark.parametrize("heads", [(8, 1, 128, "bf16"), (8, 1, 128, "f16"), (8, 2, 64, "bf16"), (4, 1, 64, "f16")])
def test_a_weight_between_two_steps_that_carries_its_row(pa, cuda_device, heads):
    """Items of more than 128 rows, weights in one 16-bit part: one token's weight is 128.5 (bf16) against a reference that
    it does not pass by enough to move it, next to the middle of two steps. Its rounding must reach numerator and
    denominator alike. (400 sequences, so that an item's tiles lie in one share.)"""
    H, G, d, t = heads
    new = 128 * G // H + 7
    b = Batch(60, [150], [new], H, G, d, t, kind="chain")
    weight = 128 * (1 + 0.98 * torch.finfo(b.dtype).eps / 2)
    b.scale = math.log(weight) / 8
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k.zero_()
    b._rows_of(b.k)[..., 0] = -48.0
    row = torch.zeros(G, d)
    b.set_row(0, 3, k=row.to(b.dtype), v=0.0)
    row[:, 0] = 8.0
    b.set_row(0, 100, k=row.to(b.dtype))
    ref = b.reference()
    half = torch.finfo(b.dtype).eps / 2
    x = repeated(b, 400, cuda_device)
    # |sum w (1 + e) v / sum w (1 + e) - out| <= half a step x sum w |v - out| / sum w (to first order in e): here
    # (|out| + weight |v - out|) / (weight + 1), and weight (v - out) = out
    check(x.run(pa), np.tile(ref, (400, 1, 1)), f"{heads}",
          allow=np.tile(2 * half * np.abs(ref) / (weight + 1), (400, 1, 1)))
    assert pa.pa_get_error() == 0


@pytest.mark.parametrize("heads", [(8, 2, 128, "bf16"), (4, 4, 64, "f32"), (4, 2, 256, "bf16"), (8, 1, 64, "bf16")])
def test_a_scale_of_zero_and_scores_of_any_size(pa, cuda_device, heads):
    """Scores of up to 1e33: a plain mean all the same (their weights are off by 2^-21 at most)."""
    H, G, d, t = heads
    b = Batch(61, [90], [30], H, G, d, t, kind="tree")
    b.q *= 1e16
    b.k *= 1e16
    b.scale = 0.0
    ref = b.reference()
    x = b.gpu(cuda_device)
    check(x.run(pa), ref, f"{heads}", allow=b.allow)
    assert pa.pa_get_error() == 0


@pytest.mark.parametrize("heads", [(8, 2, 128, "bf16"), (4, 4, 64, "f32"), (4, 2, 256, "f16"), (8, 8, 64, "bf16")])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_an_unserved_prompt_among_drafts(pa, cuda_device, heads, kind):
    """A context of 0 with more tokens than max_tree_tokens: rows of zeros, no error; the drafts beside it are right."""
    H, G, d, t = heads
    b = Batch(62, [20, 9, 0, 3000], [4, 300, 1000, 3], H, G, d, t, kind=kind)
    b.context_lens[1] = 0
    b.context_lens[2] = 0
    ref = b.reference()
    for most in (4, 64):
        out = b.gpu(cuda_device).run(pa, most=most)
        check(out, ref, f"{heads} {kind} most={most}")
        assert bool((out[4:1304] == 0).all())
        assert pa.pa_get_error() == 0
