"""GPU parity of attention over the whole range of its queries."""

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import to_host
from test_gpu_kv4 import Case as Sequences

pytestmark = pytest.mark.gpu


class Case(Sequences):
    def sizes(self):
        """max_t sum_d |q k| * scale of each row, and the largest |v| on the way."""
        group, self.vmax = self.heads // self.kv_heads, 0.0
        for b, n in enumerate(self.kv):
            for t in range(n):
                slot = int(self.table[b, t // self.page]) * self.page + t % self.page
                (kc, ks), (vc, vs) = ok.kv4_load(self.pool[self.layer], self.page, self.kv_heads, self.dim, slot)
                k, v = ok.kv4_values(kc, ks, self.k_scale), ok.kv4_values(vc, vs, self.v_scale)
                self.vmax = max(self.vmax, np.abs(v).max())
                q = self.q[int(self.start[b]):int(self.start[b + 1])].double().numpy()
                yield np.einsum("rhgd,hd->rhg", np.abs(q).reshape(-1, self.kv_heads, group, self.dim), np.abs(k)) * self.scale


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 5, 8])
@pytest.mark.parametrize("strong", [2.0 ** 20, -2.0 ** 100, 2.0 ** -80])
def test_bf16_rows_with_one_strong_channel_keep_the_others(dim, group, strong):
    """A query element far above its row's others, where every cached key is 0
    (a channel of a block that holds larger ones): the scores come from
    the other elements alone, and these keep their eight bits."""
    c = Case(dim + group, [90, 700], [3, 2], 2 * group, 2, dim, 32, "bf16")
    ratio = abs(strong) / 2.0 ** 20
    c.q[..., 5] = 0
    c.q = (c.q.double() * ratio).to(torch.bfloat16)     # (a power of two: exact)
    c.q[..., 5] = strong
    c.scale /= ratio
    page, seg = c.page, ok.kv4_segment_bytes(dim, c.page)
    view = c.pool.reshape(1, c.pages, 2, seg)
    for off in range(page):
        byte, shift, _ = ok.kv4_places(dim, page, off, False)
        view[..., byte[5]] &= np.uint8(0xF0 >> int(shift[5]))
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv", [1, 600])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_scores_up_to_their_bound(dim, kv, seed):
    """Scores of both signs up to nearly 2^26: rows stay finite, inside their values, and lse within its tolerance.
    (An fp32 score is good to no more than a few units there, so that nothing closer can be asked of the weights.)"""
    c = Case(seed * dim, [kv], [9], 4, 2, dim, 32, "bf16")
    top = max(s.max() for s in c.sizes())
    c.scale *= 0.99 * 2.0 ** 26 / top
    out, lse = (to_host(x.double()) for x in c.run())
    for rows, heads, o, l, ot, lt in c.expected():
        none = np.isneginf(l)
        assert np.isfinite(out[rows, heads]).all() and np.array_equal(np.isneginf(lse[rows, heads]), none)
        assert np.all(np.abs(out[rows, heads]) <= c.vmax * (1 + 2.0 ** -8) ** 2)
        assert np.all(np.abs(lse[rows, heads] - l)[~none] <= lt[~none])
        assert (np.abs(l[~none]) > 2.0 ** 20).any()
