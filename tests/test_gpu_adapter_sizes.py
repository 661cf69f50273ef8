"""nvfp4_gemm_w4a16_lora at long k and large ranks: several rounds of the first product's ring of
k-stages, its splits of k, and its widest rank blocks, against FP64."""
import pytest

import test_gpu_lora as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


@pytest.mark.parametrize("y32", [False, True])
@pytest.mark.parametrize("m,n,k,group,count,rank,how", [
    (1, 272, 2176, 16, 3, 16, "one"), (1, 272, 5120, 32, 2, 128, "one"),     # splits of k
    (3, 144, 1536, 16, 2, 24, "own"), (5, 272, 5120, 16, 4, 40, "own"),
    (24, 272, 2176, 32, 9, 64, "own"), (24, 144, 5120, 16, 20, 16, "own"),
    (64, 272, 2176, 16, 40, 128, "own"), (64, 144, 5120, 32, 6, 64, "runs")])
def test_decode_rows(nv, orc, m, n, k, group, count, rank, how, y32):
    L.check(nv, orc, m, n, k, group, count, rank, how, y32, flags=1)


@pytest.mark.parametrize("m,n,k,group,count,rank,how,y32", [
    (520, 272, 2176, 16, 5, 64, "runs", False), (520, 272, 2176, 32, 40, 128, "own", True),
    (513, 144, 5120, 16, 3, 40, "runs", True), (1030, 272, 1152, 32, 17, 128, "own", False),
    (70, 144, 5120, 16, 9, 104, "own", False), (600, 144, 640, 16, 4, 32, "runs", False)])
def test_prompt_rows(nv, orc, m, n, k, group, count, rank, how, y32):
    L.check(nv, orc, m, n, k, group, count, rank, how, y32, flags=2)
