"""Single tokens of windowed attention over bf16 pools keep as many bits of a weight as
paged_attention_decode: an output is off by its own rounding and little else.

Tolerance: as in test_gpu_window, but that a probability is two bf16 parts.  The first
holds 8 bits, cut off, so that what is left is below 2^-7 of the probability; it is
rounded by at most 2^-8 of itself: 2^-15.  (A second part of 2^-126 in the place of none
is far below that.)"""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_window import BF16, Case, half

pytestmark = pytest.mark.gpu


class Exact(Case):
    def reference(self, s):
        out, tol = super().reference(s)
        k, v, _ = self.rows(s)
        G = self.H // self.Hk
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        q = self.q[self.starts[s]:self.starts[s + 1]].double().transpose(0, 1)
        p = torch.softmax(q @ k.transpose(1, 2) * self.scale, dim=2)
        mass = (p @ v.abs()).transpose(0, 1)
        return out, tol - mass * (half(BF16) - 2.0 ** -15) * (1 + half(BF16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("seqs,window", [(300, 200), (3, 3000), (3, 1)])
def test_bits_of_a_weight(D, G, seqs, window):
    """Whole windows, split ones, and windows of one position."""
    lens = [1 + 53 * i % 900 if seqs > 3 else 2000 + 700 * i for i in range(seqs)]
    c = Exact([1] * seqs, lens, 2 * G, 2, D, window, 5, BF16, seed=D + G + window)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0
