"""The workspace of the cross entropy stays within what the C header says, on the host (where the library counts one SM)
and on a GPU."""
import random

import pytest

from sparse_embedding_bag_gb300 import build as B
from sparse_embedding_bag_gb300 import embbwd as E

torch = pytest.importorskip("torch")
MB = 1 << 20


@pytest.fixture(scope="module", params=["host", pytest.param("gpu", marks=pytest.mark.gpu)])
def sms(request):
    B.build()
    if request.param == "host":
        if torch.cuda.is_available():
            pytest.skip("the library counts the GPU's SMs")
        return 1
    return torch.cuda.get_device_properties(0).multi_processor_count


def bound(N, V, D, readable, gradients, sms):
    N, D = max(256, -(-N // 256) * 256), -(-D // 64) * 64
    size = N * (V // 16 + 2 * D + 16 * sms + 64)
    if not readable:
        size += 2 * V * D + 256
    if gradients:
        size += max(min(2 * N * (-(-V // 256) * 256), 512 * MB), 512 * N)
        size += max(8 * N * D, 256 * MB, 24 * 1024 * D, 256 * 1024 * sms + 1024 * D)
    return size


def test_within_the_documented_bound(sms):
    rng = random.Random(1)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    sizes = [(1, 1, 1), (1, 128256, 128), (129, 128256, 4096), (301, 50001, 1031), (4096, 128256, 4096), (1 << 20, 1 << 20, 1 << 15),
             (1, 1 << 20, 1 << 15), (256, 1 << 20, 1 << 15), (2047, 1 << 20, 8192)]
    sizes += [(spread(1, 1 << 20), spread(1, 1 << 20), spread(1, 1 << 15)) for _ in range(3000)]
    for N, V, D in sizes:
        for table in (1 << 20, (1 << 20) + 2):
            readable = D % 8 == 0 and table % 16 == 0
            for gradients in (0, 1):
                got = E.emb_cross_entropy_workspace(0, N, V, D, table, D, gradients)
                assert 0 < got <= bound(N, V, D, readable, gradients, sms), (N, V, D, table, gradients)
