"""GPU parity of attention over the whole range of its queries."""

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from test_gpu_kv4 import Case

pytestmark = pytest.mark.gpu


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
