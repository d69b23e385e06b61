"""The largest head counts, and pages that several places of the tables name."""
import pytest

from paged_util import Pages
from test_gpu_paged_cross import Cross
from test_gpu_paged_decode import Decode
from test_gpu_paged_rope import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,D", [(1024, 1, 64), (512, 2, 128), (1, 128, 256), (3, 127, 64)])
def test_decode_heads(H, G, D):
    d = Decode(Pages([70, 0, 3], H, D, "bf16", 1), G)
    d.call()
    d.check()


@pytest.mark.parametrize("H,G,D,nq", [(1024, 1, 64, 150), (1024, 1, 128, 3), (2, 128, 256, 5), (3, 127, 64, 4), (1, 65, 128, 9)])
def test_cross_heads(H, G, D, nq):
    c = Cross(Pages([70, 5], H, D, "f16", 1), [nq, 1], G)
    c.call()
    c.check()


def test_rope_heads():
    case(2, 1024, 64, 64, 64, 2, False, "bf16", seed=1)
    case(3, 1, 128, 256, 256, 4, True, "f16", seed=2, gap=8)


def test_shared_pages():
    """Two requests, and two places of one table, name the same slots."""
    pg = Pages([300, 300, 700], 2, 128, "bf16", 2)
    pg.table[1] = pg.table[0]
    pg.table[2, 6:10] = pg.table[2, :4]
    pg.keys[1], pg.values[1] = pg.keys[0], pg.values[0]
    for x in (pg.keys, pg.values):
        x[2] = x[2].clone()
        x[2][384:640] = x[2][:256]
    d = Decode(pg, 4)
    d.call()
    d.check()
    c = Cross(pg, [100, 3, 90], 4)
    c.call()
    c.check()
