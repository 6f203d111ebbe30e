"""Sums held in registers by clusters of every size (a CTA for each 2048 positions, up to 16), and the
last shapes that fit the GPU so, against the definition in 64 bits."""
import pytest
import torch

from tests.test_gpu_accumulate_weights import Case, clean_status, vsd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P_max", [4097, 9000, 12000, 12001, 16384, 20000, 25001, 30000, 32768])
@pytest.mark.parametrize("G,C", [(4, 2), (8, 2), (4, 3), (1, 16)])    # 8, 16, 12 and 16 columns
def test_held_sums_of_clusters(vsd, P_max, G, C):  # noqa: F811
    R = max(C, 4)
    rows = tuple(range(R)) if C == R else (0, R - 1) if C == 2 else (0, 1, R - 1)
    c = Case([P_max, P_max // 3, 1, P_max - 2047], P_max, R, C, G, Hkv=2, d=64, quant=(P_max + G) % 2 == 0, seed=P_max + G,
             spread=3.0, stride=P_max + (P_max % 4 and 3))
    got = c.call(vsd, rows=rows)
    c.check(got, rows)
    assert torch.equal(got, c.call(vsd, rows=rows))
    assert vsd.vsd_read_device_status() == 0


@pytest.mark.parametrize("Hkv", [9, 10])
@pytest.mark.parametrize("G", [4, 8])
def test_the_last_shape_that_is_held(vsd, Hkv, G):  # noqa: F811
    """Clusters of 16: nine fill 144 SMs; ten do not fit at once, and their slices are read again."""
    c = Case([32768], 32768, 3, 2, G, Hkv=Hkv, d=128, quant=False, seed=Hkv, spread=2.0)
    c.check(c.call(vsd), (0, 2))
    assert vsd.vsd_read_device_status() == 0
