"""Values at the ends of their ranges in decode over the 4-bit cache: a NaN that has to show however the
history is shared out. Tolerances are those of kv4_cases."""
import pytest
import torch

from kv4_cases import SCALE, PagedCase, assert_lse_close, assert_out_close, full, gauss
from oracle import oda_oracle as O
from sparse_kv_recall_b200 import build as B
from sparse_kv_recall_b200 import oda

pytestmark = pytest.mark.gpu
GROUPS = pytest.mark.parametrize("G", [1, 2, 4])


@pytest.fixture(scope="module", autouse=True)
def _library():
    B.build()
    oda.load()


def _decode(c, vis=None, scale=SCALE, dtype=torch.float32):
    out, lse = c.out(dtype, fill=3.0)
    oda.oda_kv4_decode(c.kv, full() if vis is None else vis, c.q, scale, out, c.ws, lse=lse)
    c.ok()
    return out, lse


@GROUPS
def test_a_nan_in_q_shows_however_many_ctas_share_the_history(G):
    """In its own head alone, from one CTA a (sequence, KV head) to some dozens."""
    c = PagedCase([50, 700, 3000, 20000], 2 * G, 2, seed=400)
    ref, rlse, _ = c.oracle(lambda b, t: O.full_positions(t))
    last = 2 * G - 1
    c.q[:, last, 77] = float("nan")
    out, lse = _decode(c)
    assert torch.isnan(out[:, last]).all() and torch.isnan(lse[:, last]).all()
    assert_out_close(out[:, :last], ref[:, :last])
    assert_lse_close(lse[:, :last].cpu().numpy(), rlse[:, :last])


@pytest.mark.parametrize("rows", [slice(None), slice(0, 5), slice(2990, 3000)])
def test_a_nan_in_k_shows_however_many_ctas_share_the_history(rows):
    n = 3000
    kv = [gauss((n, 1, 128), 410 + i) for i in range(2)]
    kv[0][rows, 0, 3] = float("nan")
    c = PagedCase([n], 2, 1, seed=412, rows=kv)
    out, lse = _decode(c)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
