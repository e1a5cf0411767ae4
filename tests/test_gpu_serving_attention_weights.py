"""GPU checks of gdn_paged_attention_kv8's weights one by one: light keys beside
heavy ones whose values are zero in the light ones' elements.

Key j alone has a value in element j, so element j of a row is w_j v_j: off by
2^-8 of itself for the weight's rounding to bf16, 2^-8 for the result's, and
2^-10 for scores, exponentials and sums in fp32 (bounds as in
test_gpu_serving_attention), however light the key is."""
import numpy as np
import pytest
import torch

from test_gpu_serving_attention import Case
from test_gpu_serving_attention_splits import check, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
@pytest.mark.parametrize("step", [0.55, 1.3])
@pytest.mark.parametrize("vs", [1.0, 1.7, 2.0 ** -9])
def test_light_keys_beside_heavy_ones(d, new, step, vs):
    """64 keys on four pages: weights fall by 2^-step from key to key of a page and by 2^-4step
    from page to page, value scales rise twofold."""
    c = Case(1, [(64, new), (40, 1)], 4, 2, d, 16, spread=0.0)
    c.q[...] = 0
    c.q[:, :, :2] = 1.0
    c.kq[...], c.vq[...], c.ks[...] = 0, 0, 1
    for s in range(2):
        for j in range(int(c.seq[s])):
            p, i = c.table[s, j // 16], j % 16
            c.kq[p, :, i, 0], c.kq[p, :, i, 1] = -i, -4 * (j // 16)
            c.vq[p, :, j, i], c.vs[p] = 448 if j % 3 else -11, vs * 2.0 ** (j // 16)
    c.ks, c.vs = c.ks.astype(np.float32), c.vs.astype(np.float32)
    c.scale = step * np.log(2.0)
    o = check(c, causal=False)
    assert torch.isfinite(o).all() and (o[0, 0, :64] != 0).all()
    assert (np.abs(want(c, causal=False)[0][0, 0, :64]) > 2.0 ** -60).all()
