"""GPU checks of how gdn_paged_attention_kv8 takes q: elements far below their
head's largest one, which alone make the scores, as no key has anything in
the large one's place.

Elements of at least 2^-14 of the largest are exact, so the bound of
test_gpu_serving_attention holds as it is; smaller ones are within 2^-22 of the
largest, which moves a score by up to d = 2^-22 * 448 * scale here, and a weight
by a factor of e^2d."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_serving_attention import Case, cuda
from test_gpu_serving_attention_splits import want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40], ids=["small", "large"])
@pytest.mark.parametrize("level,score", [(9, 16.0), (10, 16.0), (12, 16.0), (14, 16.0), (14, 40.0), (15, 1.0), (17, 1.0), (20, 0.25)])
@pytest.mark.parametrize("largest", [1.0, 1.9921875])
def test_small_elements_beside_a_large_one(d, new, level, score, largest):
    """Key j has its largest code in element j + 1 and a value in element j; q has
    2^-level times [1, 2) there and `largest` in element 0."""
    c = Case(level, [(48, new), (30, 1)], 4, 2, d, 16, spread=0.0)
    T = c.q.shape[0]
    q = np.zeros((T, 4, d))
    q[:, :, 1:49] = 2.0 ** -level * (1 + c.r.integers(0, 128, (T, 4, 48)) / 128) * c.r.choice([-1, 1], (T, 4, 48))
    q[:, :, 0] = largest
    c.q = cuda(q.astype(np.float32), torch.bfloat16)
    assert np.array_equal(ref.values(c.q), q)
    c.kq[...], c.vq[...], c.ks[...], c.vs[...] = 0, 0, 1, 1
    for s in range(2):
        for j in range(int(c.seq[s])):
            c.kq[c.table[s, j // 16], :, j % 16, j + 1] = 448
            c.vq[c.table[s, j // 16], :, j, j % 16] = 448
    c.scale = score * 2.0 ** level / 448
    o, w = ref.values(c.run(causal=False)), want(c, causal=False)[0]
    by = 0.0 if level <= 14 else np.expm1(2 * 2.0 ** -22 * largest * 448 * c.scale)
    bound = np.abs(w) * (2.0 ** -7 + 2.0 ** -10 + by * 1.01) + 1e-30
    assert (np.abs(o - w) <= bound).all(), "%.3g of the bound" % (np.abs(o - w) / bound).max()
